// sample.cu -- draws a token for each row of logits: temperature, top-k,
// top-p and min-p, from given uniform numbers.
//
// With m the row's largest allowed logit and r a reciprocal temperature, token
// i has the whole-number weight
//     W_i = floor(2^40 exp((l_i - m) r)),
// exp in fp32.  Sums of whole numbers do not depend on their order, so a row
// gives the same token however it is split over threads and CTAs.  Tokens are
// ranked by logit, the lower index first among equals; top-k and top-p keep a
// prefix of that ranking, i.e. all tokens above some logit tau and the first j
// of those equal to it, and min-p drops tokens of W below a bound.  The token
// drawn is the first one in index order at which the running sum of the kept
// weights passes u * total.
//
// A row takes one thread-block cluster, each CTA a slice of it.  Selecting needs
// one pass over the logits (the bound of a large batch) and no sort of the row:
//   1. every thread finds the maximum of its vectors of 16 bytes and the largest of
//      these, the cluster the row's;
//   2. a bound on how far down the kept tokens can reach.  The thread maxima
//      enter a histogram of (m - l) r in steps of 1/8: the k-th of these few
//      thousand values is at most the row's k-th, and their weights sum to no more
//      than the row's above the same logit, so the first bin that satisfies top-k
//      or top-p on them lies at or below the true cut;
//   3. the few threads whose largest vector reaches above the bound read it again
//      (from L2), those with a second one all of theirs, and list all logits above it
//      ("candidates").  The lists of all CTAs are joined in the first, the others are
//      done;
//   4. it sorts them by rank; a running sum of their weights gives how many are
//      kept; and sorts these by index, where a running sum gives the token.
// top-p without top-k needs the row's total weight: a second pass over the slice.
// Where the thread maxima do not reach the cut (a large k, a flat row with a large
// top-p) or the candidates do not fit the list, a finer histogram counts and weighs
// all tokens above the bound.  Down to the bin that holds tau they may fit after all;
// if not, the tokens of that bin alone are listed and sorted, which gives tau, and the
// token is drawn from the slices: a pass sums the weights by warps' segments, and the CTA
// and warp in whose segment the token lies find it (or, where some of tau's equals are
// left out, the CTA by visiting its slice in index order).  Where even the bin does not fit
// (thousands of equal logits), tau is found by a search over the bits of the
// (order-preserving) keys, counting and summing above trial values, two bits a round.
// Rows with neither top-k nor top-p are drawn from the slices straight away.
//
// Nothing of the row stays on chip, so that four CTAs share an SM: while one
// waits at a barrier, the others' loads keep memory busy.
//
// What bounds it: for few rows the chain of barriers and latencies, for many the
// instructions of a pass (2 a logit for the maximum, taken by vectors; some 25 for a
// weight) and of the sort, then memory.  Time of a call with 256 rows of 128,256 bf16
// logits / 8 rows of 151,936 fp32 / 1 row of 128,256 fp32, in us, where reading the
// logits once takes 9.7 / 0.7 / 0.1:
//     temperature 0 (the maximum)      19 /  9 /  9    (maximum by elements: 30 / 9 / 9)
//     top-k 50                         58 / 14 / 14
//     no rule, or min-p                84 / 16 / 12    (by visits in index order: 116 / 28 / 22)
//     top-p 0.5, some 2,000 kept      321 / 55 / 42
//     top-p 0.9, some 15,000 kept     418 / 58 / 45    (by the bit search: 1125 / 207 / 133)
//     top-k 5000                      300 / 46 / 36    (by the bit search: 1031 / 188 / 125)
// All logits equal, which the search has to settle: up to 4290 / 284 / 205.  It also
// settles rows with fewer tokens than top-k keeps (a mask that allows a dozen of them, or
// logits more than 32 nats down): 1135 / 180 / 138 with top-k 50, 1849 / 291 / 219 with
// top-p 0.9 as well (one row: of 151,936); top-p alone takes 155 / 40 / 30 there.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "step_internal.h"

namespace lbv {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;            // one thread per bin
constexpr int kList = 8 * kThreads;        // candidates the first CTA can take
constexpr int kAhead = 4;                  // vectors of a thread on their way
constexpr int kParts = 8;                  // of a warp's tokens, in the index-order sum
constexpr int kSegs = kList;               // sums of a slice's segments that are kept
constexpr int kMaxCluster = 16;
constexpr float kBinsPerNat = 8.f;
constexpr int kFine = 4 * kThreads;        // bins of a row with many candidates
constexpr float kFinePerNat = 32.f;
constexpr float kNegInf = -__builtin_huge_valf();

// Vectors of 16 bytes (and their two mask words) on the way to each thread.
struct Ring {
    uint4 v[kAhead][kThreads];
    uint32_t words[kAhead][kThreads][2];
};

// Tokens by (m - l) r in steps of 1/32: how many, and their weight.
struct Fine {
    uint64_t sum[kFine];
    unsigned count[kFine];
};

struct Shared {
    uint64_t red[3][kWarps][4];            // of reductions, by their buffer
    uint64_t all[3][kMaxCluster][4];       // one slot per CTA
    unsigned hist[kBins];
    uint64_t tops[kMaxCluster];
    uint64_t sums[kWarps];                 // drawn weight of each warp's part
    int counts[kMaxCluster];               // candidates of each CTA
    int found;                             // of this CTA so far
    unsigned scan[kWarps];
    int pick;                              // place of the drawn token
    float pick_prob;
    int bin, bin_count, above_count;       // a bin of Fine, its tokens, and what lies above
    uint64_t above_sum;
    uint64_t result[3];                    // tau, its ties, the weight down to them
    union {
        uint64_t list[kList];              // candidates: key, then the index's complement
        Fine fine;
    };
    union {
        Ring ring;                         // of the passes over the slice
        Fine merged;                       // the cluster's, between them
        uint64_t exchange[2][kList];       // of the sort's steps, after them
    };
};

// Order-preserving key of a logit (-0 made +0 before); -inf has a key above 0.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float of_key(uint32_t k)
{
    return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
}

// exp((x - top) r) in fp32, every operation rounded once; a token at the
// maximum weighs exactly 1 (the maximum may be +inf), a masked one 0 (z may be NaN
// where r is 0).
__device__ __forceinline__ float weight_f(float x, float top, float r)
{
    const float z = x == top ? 0.f : __fmul_rn(__fsub_rn(x, top), r);
    return fmaxf(expf(z), 0.f);
}

// floor(2^40 w) for 0 <= w <= 1: the significand moved to its place by shifts (a
// conversion to 64 bits takes several times longer).  NaN gives 0.
__device__ __forceinline__ uint64_t whole(float w)
{
    const uint32_t b = __float_as_uint(w), s = (b & 0x7FFFFFu) | 0x800000u;
    const uint32_t d = min(127u - (b >> 23), 63u);     // above 127: wraps, and 63 gives 0
    const uint32_t hi = s >> 15, lo = s << 17;         // 2^40 for d = 0
    const uint32_t h = d & 32u ? 0u : hi >> (d & 31u);
    const uint32_t l = d & 32u ? hi >> (d & 31u) : __funnelshift_r(lo, hi, d);
    return ((uint64_t)h << 32) | l;
}

// floor(f t / 2^24) for f <= 2^24
__device__ __forceinline__ uint64_t part(uint32_t f, uint64_t t)
{
    return (uint64_t)f * (t >> 32) * 256 + (((uint64_t)f * (t & 0xFFFFFFFFull)) >> 24);
}

__device__ __forceinline__ uint32_t fraction24(float p)
{
    const float s = p * 16777216.f;
    return s >= 16777216.f ? 16777216u : s > 0.f ? (uint32_t)s : 0u;
}

__device__ __forceinline__ uint64_t shfl_add(uint64_t v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

struct Ctx {
    Shared* sh;
    int tid, warp, lane, rank, nctas;
};

// Sums N values over the cluster's threads; every thread gets the result.  below[]
// and own[] (optional): the sums over the CTAs of lower rank, and over this one.
// buffer: another one than the last call's, unless a cluster barrier came between.
// (Functions that are not inlined take their structures by value: one whose address
// is taken lives in memory, and the passes over the logits would read it each time.)
template <int N>
__device__ __noinline__ void reduce(Ctx c, int buffer, uint64_t (&v)[N], uint64_t* below = nullptr,
                                    uint64_t* own = nullptr)
{
    Shared& sh = *c.sh;
    auto& red = sh.red[buffer];
    auto& all = sh.all[buffer];
    cg::cluster_group cl = cg::this_cluster();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = shfl_add(v[i]);
        if (c.lane == 0)
            red[c.warp][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v[i] += red[w][i];
        if (own)
            own[i] = v[i];
    }
    if (c.tid < c.nctas) {
        uint64_t* to = &cl.map_shared_rank(c.sh, c.tid)->all[buffer][c.rank][0];
#pragma unroll
        for (int i = 0; i < N; ++i)
            to[i] = v[i];
    }
    cl.sync();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint64_t t = 0, lo = 0;
        for (int r = 0; r < c.nctas; ++r) {
            lo = r == c.rank ? t : lo;
            t += all[r][i];
        }
        v[i] = t;
        if (below)
            below[i] = lo;
    }
}

template <int DT>
__device__ __forceinline__ float to_f32(uint32_t bits)     // of one element
{
    if constexpr (DT == LBV_F32)
        return __uint_as_float(bits);
    else if constexpr (DT == LBV_F16)
        return __half2float(__ushort_as_half((uint16_t)bits));
    else
        return __uint_as_float(bits << 16);
}

// A CTA's slice of the row: masked logits and NaN read as -inf, -0 as +0.
template <int DT>
struct Slice {
    static constexpr int SIZE = DT == LBV_F32 ? 4 : 2;
    static constexpr int E = 16 / SIZE;    // elements of a vector
    const unsigned char* row;              // its first element
    const uint32_t* words;                 // its mask words, or NULL
    int n;
    static __device__ __forceinline__ float clean(float v)
    {
        v = __fadd_rn(v, 0.f);
        return v != v ? kNegInf : v;
    }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t b = SIZE == 4 ? __ldg(reinterpret_cast<const uint32_t*>(row) + i)
                                     : __ldg(reinterpret_cast<const uint16_t*>(row) + i);
        return !words || ((__ldg(words + (i >> 5)) >> (i & 31)) & 1u) ? clean(to_f32<DT>(b)) : kNegInf;
    }
    // elements before the first aligned address, and up to the last
    __device__ __forceinline__ int head() const
    {
        return min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / SIZE));
    }
    __device__ __forceinline__ int tail() const { return head() + (n - head()) / E * E; }
    // a vector with the elements whose bit in m is 0 made -inf
    static __device__ __forceinline__ void hide(uint32_t (&q)[4], uint32_t m)
    {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if constexpr (DT == LBV_F32) {
                q[k] = (m >> k) & 1u ? q[k] : 0xFF800000u;
            } else {
                const uint32_t keep = ((m >> 2 * k) & 1u ? 0xFFFFu : 0u) |
                                      ((m >> (2 * k + 1)) & 1u ? 0xFFFF0000u : 0u);
                q[k] = (q[k] & keep) | ((DT == LBV_F16 ? 0xFC00FC00u : 0xFF80FF80u) & ~keep);
            }
    }
    static __device__ __forceinline__ float element(const uint32_t (&q)[4], int e)   // constant e
    {
        return DT == LBV_F32 ? clean(to_f32<DT>(q[e & 3]))
                             : clean(to_f32<DT>(e & 1 ? q[e / 2 & 3] >> 16 : q[e / 2 & 3] & 0xFFFFu));
    }
    // the largest element (NaN only if all are; the sign of a zero is open)
    static __device__ __forceinline__ float largest(const uint32_t (&q)[4])
    {
        if constexpr (DT == LBV_F32) {
            return fmaxf(fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1])),
                         fmaxf(__uint_as_float(q[2]), __uint_as_float(q[3])));
        } else if constexpr (DT == LBV_F16) {
            __half2 h[4];
            memcpy(h, q, 16);
            const __half2 v = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(v), __high2float(v));
        } else {
            __nv_bfloat162 h[4];
            memcpy(h, q, 16);
            const __nv_bfloat162 v = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(v), __high2float(v));
        }
    }
};

__device__ __forceinline__ void copy_async(void* to, const void* from, int bytes)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(to);
    if (bytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(d), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(d), "l"(from) : "memory");
}

// Calls vec(words, first index) for the thread's vectors of the slice, and one(value,
// index) for a logit before the first aligned address or after the last; indexes
// ascend, but for that the ones come first and last.  16-byte copies, several of them in
// flight, go into places of the ring that only this thread reads (in registers, a
// rotation of the buffers would wait for the copy that was just asked for).
template <int DT, typename V, typename F>
__device__ __forceinline__ void each_vector(const Slice<DT>& s, int tid, Ring& ring, V vec, F one)
{
    constexpr int SIZE = Slice<DT>::SIZE, E = Slice<DT>::E;
    const int head = s.head(), body = (s.n - head) / E, tail = head + body * E;
    const uint4* v = reinterpret_cast<const uint4*>(s.row + head * SIZE);
    auto ask = [&](int i, int st) {
        if (i < body) {
            copy_async(&ring.v[st][tid], v + i, 16);
            if (s.words) {
                const int d = head + i * E;
                copy_async(&ring.words[st][tid][0], s.words + (d >> 5), 4);
                copy_async(&ring.words[st][tid][1], s.words + ((d + E - 1) >> 5), 4);
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll 1
    for (int u = 0; u < kAhead; ++u)
        ask(tid + u * kThreads, u);
    if (tid < head)
        one(s.get(tid), tid);
    int st = 0;
#pragma unroll 1
    for (int i = tid; i < body; i += kThreads) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead - 1) : "memory");
        const uint4 w = ring.v[st][tid];
        const int d = head + i * E;
        uint32_t q[4] = {w.x, w.y, w.z, w.w};
        if (s.words)
            s.hide(q, __funnelshift_r(ring.words[st][tid][0], ring.words[st][tid][1], d & 31));
        ask(i + kAhead * kThreads, st);
        st = st + 1 == kAhead ? 0 : st + 1;
        vec(q, d);
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    if (tail + tid < s.n)                  // fewer than E of them
        one(s.get(tail + tid), tail + tid);
}

// Calls f(value, index) for the thread's logits of the slice, two of a vector unrolled.
template <int DT, typename F>
__device__ __forceinline__ void each(const Slice<DT>& s, int tid, Ring& ring, F f)
{
    each_vector(s, tid, ring, [&](uint32_t (&q)[4], int d) {
#pragma unroll 1
        for (int e = 0; e < Slice<DT>::E; e += 2) {
            uint32_t two[4];
            if constexpr (DT == LBV_F32) {
                two[0] = e ? q[2] : q[0];
                two[1] = e ? q[3] : q[1];
            } else {
                two[0] = e < 4 ? (e < 2 ? q[0] : q[1]) : (e < 6 ? q[2] : q[3]);
            }
            f(s.element(two, 0), d + e);
            f(s.element(two, 1), d + e + 1);
        }
    }, f);
}

// The sum of whole(f(value)) over the thread's logits.  f gives 0 to 1; adding a power
// of two, rounded towards zero, leaves the integer part of 2^17 f in the low bits of the
// sum, and that of 2^40 times the remainder in those of a second one; their biases are
// taken off once a vector.  seg (optional): the sum over each warp's vectors of a round, in
// index order, for the first kSegs rounds and warps.
template <int DT, typename F>
__device__ __forceinline__ uint64_t sum_whole(const Slice<DT>& s, int tid, Ring& ring, uint64_t* seg, F f)
{
    constexpr int E = Slice<DT>::E;
    constexpr uint32_t kHigh = 0x42800000u, kLow = 0x37000000u;        // 2^6, 2^-17
    uint64_t sum = 0;
    int at = tid >> 5, rest = (s.n - s.head()) / E - (tid & ~31);      // the warp's segment; vectors from its first on
    each_vector(s, tid, ring, [&](uint32_t (&q)[4], int) {
        uint32_t high = 0, low = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float w = f(s.element(q, e));
            const float a = __fadd_rz(w, __uint_as_float(kHigh));
            const float over = __fsub_rn(w, __fsub_rn(a, __uint_as_float(kHigh)));
            high += __float_as_uint(a);
            low += __float_as_uint(__fadd_rz(over, __uint_as_float(kLow)));
        }
        high -= E * kHigh, low -= E * kLow;
        sum += ((uint64_t)high << 23) + low;
        if (seg) {                                                     // 2^20 and 2^26 a lane at most
            const unsigned lanes = rest >= 32 ? 0xffffffffu : (1u << rest) - 1;
            high = __reduce_add_sync(lanes, high), low = __reduce_add_sync(lanes, low);
            if ((tid & 31) == 0 && at < kSegs)
                seg[at] = ((uint64_t)high << 23) + low;
            at += kWarps, rest -= kThreads;
        }
    }, [&](float x, int) { sum += whole(f(x)); });
    return sum;
}

struct Row {
    float top, filter_r, draw_r, min_p, top_p;
    int k;                                 // 0: off
    float u;
};

// Kept tokens: key above tau, or the first `ties` in index order equal to it.
struct Kept {
    uint32_t tau;
    uint64_t ties;
};

// The largest key t for which test(t, sum of f over the tokens with key >= t)
// holds; it holds at 0.  f(x) is a count or a weight, test is monotone in t.
template <typename D, typename F, typename Test>
__device__ __forceinline__ uint32_t search(Ctx c, const D& d, F f, Test test)
{
    uint32_t t = 0;
    for (int bit = 30; bit >= 0; bit -= 2) {
        uint64_t s1 = 0, s2 = 0, s3 = 0;
        const uint32_t t1 = t | (1u << bit), t2 = t | (2u << bit), t3 = t | (3u << bit);
        each(d, c.tid, c.sh->ring, [&](float x, int) {
            const uint32_t k = key_of(x);
            if (k >= t1) {
                const uint64_t w = f(x);
                s1 += w;
                s2 += k >= t2 ? w : 0;
                s3 += k >= t3 ? w : 0;
            }
        });
        uint64_t v[3] = {s1, s2, s3};
        reduce<3>(c, (bit >> 1) & 1, v);
        t = test(t3, v[2]) ? t3 : test(t2, v[1]) ? t2 : test(t1, v[0]) ? t1 : t;
    }
    return t;
}

// tau and its ties by search.  total: the weight of the whole row (without top-k).
template <typename D>
__device__ __noinline__ Kept select(Ctx c, D d, Row row, uint64_t total)
{
    Kept kept = {0u, ~0ull};
    uint32_t tau_k = 0;
    auto weight = [&](float x) { return whole(weight_f(x, row.top, row.filter_r)); };
    if (row.k > 0) {
        const uint64_t k = (uint64_t)row.k;
        tau_k = search(c, d, [](float) { return (uint64_t)1; },
                       [&](uint32_t, uint64_t n) { return n >= k; });
        // what lies above it
        uint64_t n = 0, sum = 0;
        each(d, c.tid, c.sh->ring, [&](float x, int) {
            if (key_of(x) > tau_k) {
                n += 1;
                sum += weight(x);
            }
        });
        uint64_t v[2] = {n, sum};
        reduce<2>(c, 2, v);                            // a search uses 1, 0, ..., 1, 0
        kept.tau = tau_k;
        kept.ties = k - v[0];
        total = v[1] + kept.ties * weight(of_key(tau_k));    // a masked tau weighs 0
    }
    if (row.top_p < 1.f) {
        const uint64_t limit = part(fraction24(row.top_p), total);
        if (limit == 0)
            return Kept{key_of(row.top), 1};
        const uint32_t tau = search(c, d, weight, [&](uint32_t t, uint64_t s) {
            return t <= tau_k || s >= limit;
        });
        uint64_t sum = 0;
        each(d, c.tid, c.sh->ring, [&](float x, int) { sum += key_of(x) > tau ? weight(x) : 0; });
        uint64_t v[1] = {sum};
        reduce<1>(c, 1, v);
        const uint64_t w = weight(of_key(tau));
        const uint64_t j = w ? (limit - v[0] + w - 1) / w : 1;
        kept.ties = tau == tau_k && j > kept.ties ? kept.ties : j;
        kept.tau = tau;
    }
    cg::this_cluster().sync();                         // every buffer is free again
    return kept;
}

// The block's sum of v, and in `before` that of the threads before this one.
__device__ __noinline__ uint64_t block_scan(Ctx c, uint64_t v, uint64_t& before)
{
    uint64_t upto = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, upto, s);
        upto += c.lane >= s ? o : 0;
    }
    __syncthreads();
    if (c.lane == 31)
        c.sh->sums[c.warp] = upto;
    __syncthreads();
    uint64_t all = 0, below = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        below = i == c.warp ? all : below;
        all += c.sh->sums[i];
    }
    before = below + upto - v;
    return all;
}

// Draws from the kept tokens of all slices in index order: one pass gives each CTA's
// weight, and the CTA in which the running sum passes u's share looks for the token.
// Returns its place in the slice, or -1 in the other CTAs; *prob its probability
// among the kept ones.
template <int DT>
__device__ __noinline__ int draw(Ctx c, Slice<DT> d, Row row, Kept kept, float* prob)
{
    Shared& sh = *c.sh;
    auto share = [&](float x) {            // of a token that the ranking keeps
        const float w = weight_f(x, row.top, row.draw_r);
        const float f = row.filter_r == row.draw_r || row.min_p <= 0.f ? w : weight_f(x, row.top, row.filter_r);
        return f >= row.min_p || row.min_p <= 0.f ? w : 0.f;
    };
    auto weight = [&](float x) { return whole(share(x)); };
    // all of tau's are kept, or those above it and some of its own
    const bool ties_out = kept.ties != ~0ull;
    const float tau = kept.tau ? of_key(kept.tau) : kNegInf, from = ties_out ? of_key(kept.tau + 1) : tau;
    auto kept_weight = [&](float x) { return x >= from ? weight(x) : 0; };
    unsigned equal = 0;
    uint64_t sum = sum_whole(d, c.tid, sh.ring, sh.list, [&](float x) {
        equal += ties_out && x == tau;
        return x >= from ? share(x) : 0.f;
    });
    uint64_t all[2] = {sum, equal}, below[2], here[2];
    reduce<2>(c, 2, all, below, here);
    const uint64_t tie_w = all[1] ? weight(of_key(kept.tau)) : 0;
    const uint64_t ties_below = min(kept.ties, below[1]), ties_upto = min(kept.ties, below[1] + here[1]);
    const uint64_t total = all[0] + min(kept.ties, all[1]) * tie_w;
    uint64_t at = below[0] + ties_below * tie_w;
    uint32_t f = fraction24(row.u);
    f = f > 16777215u ? 16777215u : f;
    const uint64_t target = part(f, total);
    if (target < at || target >= at + here[0] + (ties_upto - ties_below) * tie_w)
        return -1;
    // ---- by the segments' sums, where ties need no count ----
    const int head = d.head(), body = (d.n - head) / Slice<DT>::E;
    const int segs = (body + kThreads - 1) / kThreads * kWarps;
    if (!ties_out && segs <= kSegs) {
        uint64_t first = at, before;
        if (head > 0)
            first += block_scan(c, c.tid < head ? kept_weight(d.get(c.tid)) : 0, before);
        const int each_of = (segs + kThreads - 1) / kThreads, s0 = c.tid * each_of, s1 = min(s0 + each_of, segs);
        auto seg = [&](int i) { return i / kWarps * kThreads + i % kWarps * 32 < body ? sh.list[i] : 0; };
        uint64_t mine = 0;
        for (int i = s0; i < s1; ++i)
            mine += seg(i);
        if (c.tid == 0)
            sh.bin = sh.pick = -1;
        const uint64_t sums = block_scan(c, mine, before);       // its barriers order sh.bin and the segments
        before += first;
        if (target >= before && target < before + mine)
            for (int i = s0; i < s1; ++i) {
                const uint64_t w = seg(i);
                if (target < before + w) {
                    sh.bin = i;
                    sh.above_sum = before;
                    break;
                }
                before += w;
            }
        __syncthreads();
        if (target >= first && target < first + sums) {          // else in the few logits around them
            if (c.warp == 0) {
                constexpr int E = Slice<DT>::E;
                const int v = sh.bin / kWarps * kThreads + sh.bin % kWarps * 32 + c.lane, i0 = head + v * E;
                float x[E];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[e] = v < body ? d.get(i0 + e) : kNegInf;
                uint64_t w[E], mine = 0;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    w[e] = kept_weight(x[e]);
                    mine += w[e];
                }
                uint64_t upto = mine;
#pragma unroll
                for (int s = 1; s < 32; s <<= 1) {
                    const uint64_t o = __shfl_up_sync(0xffffffffu, upto, s);
                    upto += c.lane >= s ? o : 0;
                }
                uint64_t here = sh.above_sum + upto - mine;
                if (target >= here && target < here + mine)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (target >= here && target < here + w[e]) {
                            sh.pick = i0 + e;
                            sh.pick_prob = __fdiv_rn(__ull2float_rn(w[e]), __ull2float_rn(total));
                        }
                        here += w[e];
                    }
            }
            __syncthreads();
            *prob = sh.pick_prob;
            return sh.pick;
        }
    }
    // ---- by visits in index order ----
    const int groups = (d.n + 31) / 32, per = (groups + kWarps - 1) / kWarps;
    const int g0 = min(c.warp * per, groups), g1 = min(g0 + per, groups);
    const unsigned before = (1u << c.lane) - 1;
    // ties in index order ahead of this warp
    uint64_t tie_base = below[1];
    if (kept.ties < all[1]) {
        unsigned mine = 0;
#pragma unroll 8
        for (int g = g0; g < g1; ++g) {
            const int i = g * 32 + c.lane;
            mine += i < d.n && key_of(d.get(i)) == kept.tau;
        }
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (c.lane == 0)
            sh.scan[c.warp] = mine;
        __syncthreads();
        for (int w = 0; w < c.warp; ++w)
            tie_base += sh.scan[w];
    }
    // visits groups [a, b) of the warp's in index order, `ties` of tau's before them:
    // f(place, weight) by all lanes
    auto visit = [&](int a, int b, uint64_t& ties, auto f) {
#pragma unroll 8
        for (int g = a; g < b; ++g) {
            const int i = g * 32 + c.lane;
            const float x = i < d.n ? d.get(i) : kNegInf;
            const uint32_t k = key_of(x);
            const bool tie = i < d.n && k == kept.tau;
            const unsigned tied = __ballot_sync(0xffffffffu, tie);
            const bool in = k > kept.tau || (tie && ties + __popc(tied & before) < kept.ties);
            ties += __popc(tied);
            if (f(i, in ? weight(x) : 0))
                return;
        }
    };
    // the weight of the warp's tokens, by parts, with the ties before each
    const int step = (g1 - g0 + kParts - 1) / kParts;
    uint64_t ties = tie_base, my_sum = 0, my_ties = 0;              // of part `lane`
    sum = 0;
    for (int q = 0; q < kParts; ++q) {
        const int a = min(g0 + q * step, g1), b = min(a + step, g1);
        my_ties = c.lane == q ? ties : my_ties;
        uint64_t s = 0;
        visit(a, b, ties, [&](int, uint64_t w) { s += w; return false; });
        s = shfl_add(s);
        my_sum = c.lane == q ? s : my_sum;
        sum += s;
    }
    if (c.lane == 0)
        sh.sums[c.warp] = sum;
    if (c.tid == 0)
        sh.pick = -1;
    __syncthreads();
    for (int w = 0; w < c.warp; ++w)
        at += sh.sums[w];
    if (target >= at && target < at + sum) {
        int q = 0;
        uint64_t s = __shfl_sync(0xffffffffu, my_sum, 0);
        while (target >= at + s) {
            at += s;
            s = __shfl_sync(0xffffffffu, my_sum, ++q);
        }
        ties = __shfl_sync(0xffffffffu, my_ties, q);
        const int a = min(g0 + q * step, g1), b = min(a + step, g1);
        visit(a, b, ties, [&](int i, uint64_t w) {
            uint64_t upto = w;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const uint64_t o = __shfl_up_sync(0xffffffffu, upto, s);
                upto += c.lane >= s ? o : 0;
            }
            const unsigned past = __ballot_sync(0xffffffffu, at + upto > target);
            if (past == 0) {
                at += __shfl_sync(0xffffffffu, upto, 31);
                return false;
            }
            if (c.lane == __ffs(past) - 1) {
                sh.pick = i;
                sh.pick_prob = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(total));
            }
            return true;
        });
    }
    __syncthreads();
    *prob = sh.pick_prob;
    return sh.pick;
}

// Sorts list[0 .. kThreads E) (or a smaller power of two n2, E = 1) in descending order,
// bitonic, E elements a thread in registers (thread t: t, t + kThreads, ...): exchanges
// over strides below 32 by shuffles, over kThreads and more within the thread, and those
// between through shared memory.
template <int E>
__device__ __noinline__ void sort_list(Shared& sh, int n2, int tid)
{
    uint64_t v[E];
#pragma unroll
    for (int q = 0; q < E; ++q)
        v[q] = E > 1 || tid < n2 ? sh.list[tid + q * kThreads] : 0;
    int half = 0;
#pragma unroll 1
    for (int size = 2; size <= n2; size *= 2)
#pragma unroll 1
        for (int stride = size / 2; stride > 0; stride /= 2) {
            uint64_t o[E];
            if (stride < 32) {
#pragma unroll
                for (int q = 0; q < E; ++q)
                    o[q] = __shfl_xor_sync(0xffffffffu, v[q], stride);
            } else if (E == 1 || stride < kThreads) {
                uint64_t* x = sh.exchange[half];
                half ^= 1;                         // one barrier a step
#pragma unroll
                for (int q = 0; q < E; ++q)
                    x[tid + q * kThreads] = v[q];
                __syncthreads();
#pragma unroll
                for (int q = 0; q < E; ++q)
                    o[q] = x[(tid ^ stride) + q * kThreads];
            } else {
#pragma unroll
                for (int q = 0; q < E; ++q)
                    o[q] = stride == kThreads       ? v[q ^ (E > 1 ? 1 : 0)]
                           : stride == 2 * kThreads ? v[q ^ (E > 2 ? 2 : 0)]
                                                    : v[q ^ (E > 4 ? 4 : 0)];
            }
#pragma unroll
            for (int q = 0; q < E; ++q) {
                const int i = tid + q * kThreads;
                const bool larger = ((i & stride) == 0) == ((i & size) == 0);
                v[q] = (v[q] > o[q]) == larger ? v[q] : o[q];
            }
        }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < E; ++q)
        if (E > 1 || tid < n2)
            sh.list[tid + q * kThreads] = v[q];
    __syncthreads();
}

__device__ __forceinline__ void sort_list(Shared& sh, int n2, int tid)
{
    if (n2 <= kThreads)
        sort_list<1>(sh, n2, tid);
    else if (n2 == 2 * kThreads)
        sort_list<2>(sh, n2, tid);
    else if (n2 == 4 * kThreads)
        sort_list<4>(sh, n2, tid);
    else
        sort_list<8>(sh, n2, tid);
}

__device__ __forceinline__ int power_above(int n)
{
    return n <= 2 ? 2 : 1 << (32 - __clz(n - 1));
}

// Lists in the first CTA the tokens that visit(found) finds in each slice; returns
// their number, and lists nothing where they are more than fit.
template <typename Visit>
__device__ __forceinline__ int gather(Ctx c, int begin, Visit visit)
{
    Shared& sh = *c.sh;
    cg::cluster_group cl = cg::this_cluster();
    visit([&](float x, int i) {
        const int at = atomicAdd(&sh.found, 1);
        if (at < kList)
            sh.list[at] = ((uint64_t)key_of(x) << 32) | (0xFFFFFFFFu - (uint32_t)(begin + i));
    });
    __syncthreads();
    const int here = sh.found;
    if (c.tid < c.nctas)
        cl.map_shared_rank(&sh, c.tid)->counts[c.rank] = here;
    cl.sync();
    int n = 0, before = 0;
    for (int r = 0; r < c.nctas; ++r) {
        before = r == c.rank ? n : before;
        n += sh.counts[r];
    }
    if (n <= kList) {
        Shared* to = cl.map_shared_rank(&sh, 0);
        if (c.rank > 0)
            for (int i = c.tid; i < here; i += kThreads)
                to->list[before + i] = sh.list[i];
        cl.sync();
    }
    return n;
}

// For a row with many candidates, all of them >= cut.  Returns kSearch where the finer
// histogram does not resolve it, kByValue with tau and its ties, or the number of
// candidates where, with the finer bound, they fit the list after all.
// total: the weight of the whole row (without top-k).
constexpr int kSearch = -2, kByValue = -1;

template <int DT>
__device__ __noinline__ int select_binned(Ctx c, Slice<DT> slice, Row row, float cut,
                                          uint64_t total, int begin, Kept& kept)
{
    Shared& sh = *c.sh;
    cg::cluster_group cl = cg::this_cluster();
    const bool by_sum = row.top_p < 1.f;
    const float scale = row.filter_r * kFinePerNat;
    auto bin_of = [&](float v) {                       // below the cut: none of the bins
        const float b = v == row.top ? 0.f : (row.top - v) * scale;
        return v >= cut && b < (float)kFine ? (int)b : kFine;
    };
    for (int i = c.tid; i < kFine; i += kThreads) {
        sh.fine.sum[i] = 0;
        sh.fine.count[i] = 0;
    }
    __syncthreads();
    each(slice, c.tid, sh.ring, [&](float x, int) {
        const int b = bin_of(x);
        if (b < kFine) {
            atomicAdd(&sh.fine.count[b], 1u);
            const uint64_t w = by_sum ? whole(weight_f(x, row.top, row.filter_r)) : 0;
            if (w)
                atomicAdd(reinterpret_cast<unsigned long long*>(&sh.fine.sum[b]), (unsigned long long)w);
        }
    });
    // Each CTA merges its share of the bins (nctas is a power of two): neighbouring
    // lanes read a bin of all CTAs, and hand each the sum.
    __syncthreads();
    cl.sync();
    {
        Shared* peer = cl.map_shared_rank(&sh, c.tid & (c.nctas - 1));
        uint64_t s[4];
        unsigned n[4];
        int b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            b[q] = (c.rank * kFine + q * kThreads + c.tid) / c.nctas;
            s[q] = peer->fine.sum[b[q]];
            n[q] = peer->fine.count[b[q]];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            for (int d = c.nctas / 2; d > 0; d >>= 1) {
                s[q] += __shfl_xor_sync(0xffffffffu, s[q], d);
                n[q] += __shfl_xor_sync(0xffffffffu, n[q], d);
            }
            peer->merged.sum[b[q]] = s[q];
            peer->merged.count[b[q]] = n[q];
        }
    }
    cl.sync();
    // this thread's four bins, and what lies above them
    uint64_t sums[4], sum_at, count_at;
    unsigned counts[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        sums[q] = sh.merged.sum[4 * c.tid + q];
        counts[q] = sh.merged.count[4 * c.tid + q];
    }
    block_scan(c, (sums[0] + sums[1]) + (sums[2] + sums[3]), sum_at);
    block_scan(c, (counts[0] + counts[1]) + (counts[2] + counts[3]), count_at);
    // the bin in which the running count (or weight) reaches `want`
    auto locate = [&](bool by_count, uint64_t want) {
        __syncthreads();
        if (c.tid == 0)
            sh.bin = -1;
        __syncthreads();
        uint64_t n = count_at, s = sum_at;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint64_t from = by_count ? n : s, to = by_count ? n + counts[q] : s + sums[q];
            if (from < want && want <= to) {
                sh.bin = 4 * c.tid + q;
                sh.bin_count = (int)counts[q];
                sh.above_count = (int)n;
                sh.above_sum = s;
            }
            n += counts[q];
            s += sums[q];
        }
        __syncthreads();
        return sh.bin;
    };
    // the tokens of bins [b0, b1] into the first CTA's list
    auto list_bins = [&](int b0, int b1) {
        return gather(c, begin, [&](auto found) {
            each(slice, c.tid, sh.ring, [&](float x, int i) {
                const int b = bin_of(x);
                if (b >= b0 && b <= b1)
                    found(x, i);
            });
        });
    };
    // tau by the tokens of a bin in order of rank: the first `most` of them, or as
    // many as bring the weight from `above` up to `limit`
    int listed = -1;
    auto resolve = [&](int bin, int n, uint64_t above, int most, uint64_t limit) {
        if (c.tid == 0)
            sh.found = 0;
        cl.sync();                                     // the last results have been read
        if (bin != listed)
            list_bins(bin, bin);
        if (c.rank == 0) {
            if (bin != listed) {
                const int n2 = power_above(n);
                for (int i = n + c.tid; i < n2; i += kThreads)
                    sh.list[i] = 0;
                __syncthreads();
                sort_list(sh, n2, c.tid);
            }
            const int per = (most + kThreads - 1) / kThreads, i0 = c.tid * per, i1 = min(i0 + per, most);
            uint64_t mine = 0, at;
            for (int i = i0; i < i1; ++i)
                mine += whole(weight_f(of_key((uint32_t)(sh.list[i] >> 32)), row.top, row.filter_r));
            const uint64_t all = block_scan(c, mine, at);
            if (c.tid == 0)
                sh.pick = most;
            __syncthreads();
            at += above;
            if (at < limit && limit <= at + mine)
                for (int i = i0; i < i1; ++i) {
                    at += whole(weight_f(of_key((uint32_t)(sh.list[i] >> 32)), row.top, row.filter_r));
                    if (at >= limit) {
                        sh.pick = i + 1;
                        break;
                    }
                }
            __syncthreads();
            const int taken = sh.pick;
            const uint32_t tau = (uint32_t)(sh.list[taken - 1] >> 32);
            uint64_t counts = 0, unused;               // above tau, and equal to it
            for (int i = c.tid; i < n; i += kThreads) {
                const uint32_t k = (uint32_t)(sh.list[i] >> 32);
                counts += (k > tau ? 1 : 0) + ((uint64_t)(k == tau) << 32);
            }
            counts = block_scan(c, counts, unused);
            const uint64_t ties = (uint64_t)taken - (counts & 0xFFFFFFFFu);
            if (c.tid < c.nctas) {
                Shared* o = cl.map_shared_rank(&sh, c.tid);
                o->result[0] = tau;
                o->result[1] = ties == counts >> 32 ? ~0ull : ties;
                o->result[2] = above + all;
            }
        }
        listed = bin;
        cl.sync();
        kept.tau = (uint32_t)sh.result[0];
        kept.ties = sh.result[1];
    };
    // So many candidates are sorted in less time than drawing from the slices takes: with the
    // larger clusters of a few rows (8 rows of 151,936 fp32, 2,000 candidates: 80 us sorted, 55
    // from the slices), and with the smaller ones (256 rows of 128,256 bf16: 321 and 362).
    const int sorted = c.nctas > 8 ? 2 * kThreads : kList;
    // Below a cut that min-p gave neither top-k nor top-p need be reached: then min-p
    // alone decides, and all tokens are kept here.
    const int unreached = cut > kNegInf ? kByValue : kSearch;
    int bin_k = kFine, count_k = 0, need = 0;
    uint64_t above_k = 0;
    auto list_down_to = [&](int bin) {
        if (c.tid == 0)
            sh.found = 0;
        cl.sync();                                     // the histograms have been read
        return list_bins(0, bin);
    };
    if (row.k > 0) {
        bin_k = locate(true, (uint64_t)row.k);
        if (bin_k < 0)
            return unreached;
        count_k = sh.bin_count;
        above_k = sh.above_sum;
        need = row.k - sh.above_count;
        if (sh.above_count + count_k <= sorted)
            return list_down_to(bin_k);
        if (count_k > kList)
            return kSearch;
        resolve(bin_k, count_k, above_k, need, ~0ull);
        total = sh.result[2];
    }
    if (by_sum) {
        const uint64_t limit = part(fraction24(row.top_p), total);
        if (limit == 0) {
            kept = Kept{key_of(row.top), 1};
            return kByValue;
        }
        const int bin = locate(false, limit);
        if (bin < 0)
            return unreached;
        const int count = sh.bin_count;
        if (row.k == 0 && sh.above_count + count <= sorted)
            return list_down_to(bin);
        if (count > kList)
            return kSearch;
        if (bin < bin_k)
            resolve(bin, count, sh.above_sum, count, limit);
        else
            resolve(bin_k, count_k, above_k, need, limit);
    }
    return kByValue;
}

// Draws from the n candidates of the list, of which every kept token is one.
// total: the weight of the whole row (without top-k).
__device__ __forceinline__ void draw_listed(Ctx c, const Row& row, bool by_sum, uint64_t total, int n,
                                            const SampleParams& p, int m)
{
    Shared& sh = *c.sh;
    uint64_t* list = sh.list;
    int n2 = power_above(n);
    for (int i = n + c.tid; i < n2; i += kThreads)
        list[i] = 0;
    __syncthreads();
    sort_list(sh, n2, c.tid);
    // ---- how many are kept: a prefix of the ranking ----
    const int most = row.k > 0 ? min(row.k, n) : n;
    int per = (most + kThreads - 1) / kThreads, i0 = c.tid * per, i1 = min(i0 + per, most);
    uint64_t limit = ~0ull, at = 0;
    if (by_sum) {
        uint64_t mine = 0;
        for (int i = i0; i < i1; ++i)
            mine += whole(weight_f(of_key((uint32_t)(list[i] >> 32)), row.top, row.filter_r));
        const uint64_t all = block_scan(c, mine, at);
        limit = part(fraction24(row.top_p), row.k > 0 ? all : total);
    }
    int kept = 0;
    for (int i = i0; i < i1; ++i) {
        const float w = weight_f(of_key((uint32_t)(list[i] >> 32)), row.top, row.filter_r);
        kept += (i == 0 || at < limit) && w >= row.min_p;
        at += by_sum ? whole(w) : 0;
    }
    uint64_t unused;
    kept = (int)block_scan(c, (uint64_t)kept, unused);
    // ---- these by index ----
    n2 = power_above(kept);
    __syncthreads();
    for (int i = c.tid; i < n2; i += kThreads)
        list[i] = i < kept ? (list[i] << 32) | (list[i] >> 32) : 0;
    __syncthreads();
    sort_list(sh, n2, c.tid);
    per = (kept + kThreads - 1) / kThreads, i0 = c.tid * per, i1 = min(i0 + per, kept);
    uint64_t mine = 0;
    for (int i = i0; i < i1; ++i)
        mine += whole(weight_f(of_key((uint32_t)list[i]), row.top, row.draw_r));
    const uint64_t all = block_scan(c, mine, at);
    uint32_t f = fraction24(row.u);
    f = f > 16777215u ? 16777215u : f;
    const uint64_t target = part(f, all);
    if (at <= target && target < at + mine)
        for (int i = i0; i < i1; ++i) {
            const uint64_t w = whole(weight_f(of_key((uint32_t)list[i]), row.top, row.draw_r));
            if (at <= target && target < at + w) {
                p.token[m] = (int)(0xFFFFFFFFu - (uint32_t)(list[i] >> 32));
                if (p.prob)
                    p.prob[m] = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(all));
            }
            at += w;
        }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 4) lbv_sample_kernel(const __grid_constant__ SampleParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    cg::cluster_group cl = cg::this_cluster();
    Ctx c;
    c.sh = &sh;
    c.tid = threadIdx.x;
    c.warp = c.tid >> 5;
    c.lane = c.tid & 31;
    c.nctas = p.ctas;
    c.rank = blockIdx.x % p.ctas;
    const int m = blockIdx.x / p.ctas;
    after_previous();
    const int begin = min(c.rank * p.slice, p.N);

    Slice<DT> slice;
    slice.n = min(p.slice, p.N - begin);
    slice.row = static_cast<const unsigned char*>(p.logits) +
                ((int64_t)m * p.ld + begin) * Slice<DT>::SIZE;
    slice.words = p.mask ? p.mask + (int64_t)m * p.mask_ld + begin / 32 : nullptr;
    Row row;
    const float t = p.temperature ? p.temperature[m] : 1.f;
    row.u = p.u[m];
    row.k = p.top_k ? p.top_k[m] : 0;
    row.top_p = p.top_p ? p.top_p[m] : 1.f;
    row.min_p = p.min_p ? p.min_p[m] : 0.f;
    const bool greedy = !(t > 0.f) || !(row.min_p <= 1.f);
    row.draw_r = __frcp_rn(t);
    row.filter_r = p.temperature_last ? 1.f : row.draw_r;

    cl.barrier_arrive();                               // waited for before the first remote store

    // ---- the thread's and the row's first maximum ----
    // (by vectors: the largest and the next largest of their maxima)
    float high = kNegInf, next = kNegInf;
    int high_at = 0;
    auto higher = [&](float v, int i) {
        next = fmaxf(next, fminf(v, high));
        high_at = v > high ? i : high_at;
        high = fmaxf(high, v);
    };
    each_vector(slice, c.tid, sh.ring, [&](uint32_t (&q)[4], int d) { higher(slice.largest(q), d); },
                higher);
    high = __fadd_rn(high, 0.f);                       // -0 to +0
    sh.hist[c.tid] = 0;
    if (c.tid == 0)
        sh.found = 0;
    uint64_t best = 0;
    if (slice.n > 0)                                   // a row of -inf has a key above 0 too
        best = ((uint64_t)key_of(high) << 32) | (0xFFFFFFFFu - (uint32_t)(begin + high_at));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, best, s);
        best = o > best ? o : best;
    }
    if (c.lane == 0)
        sh.red[0][c.warp][0] = best;
    __syncthreads();
    cl.barrier_wait();
    if (c.tid < c.nctas) {
        uint64_t b = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            b = sh.red[0][w][0] > b ? sh.red[0][w][0] : b;
        cl.map_shared_rank(&sh, c.tid)->tops[c.rank] = b;
    }
    cl.sync();
    best = 0;
    for (int r = 0; r < c.nctas; ++r)
        best = sh.tops[r] > best ? sh.tops[r] : best;
    row.top = of_key((uint32_t)(best >> 32));
    const int first = (int)(0xFFFFFFFFu - (uint32_t)best);
    if (best == 0 || row.top == kNegInf || greedy) {   // nothing allowed, or the maximum itself
        const Slice<DT> all = {slice.row - (int64_t)begin * Slice<DT>::SIZE,
                               slice.words ? slice.words - begin / 32 : nullptr, p.N};
        const int i = first + c.lane;                  // the first of its vector
        if (c.rank == 0 && c.warp == 0) {
            const bool none = best == 0 || row.top == kNegInf;
            const unsigned at = __ballot_sync(0xffffffffu, i >= 0 && i < p.N && all.get(i) == row.top);
            if (c.lane == 0) {
                p.token[m] = none ? -1 : first + __ffs(at) - 1;
                if (p.prob)
                    p.prob[m] = none ? 0.f : 1.f;
            }
        }
        return;
    }

    Kept kept = {0u, ~0ull};
    const bool by_rank = row.k > 0 && row.k < p.N, by_sum = row.top_p < 1.f;
    row.k = by_rank ? row.k : 0;
    if (by_rank || by_sum) {
        // ---- the histogram, and with it the row's weight ----
        const float scale = row.filter_r * kBinsPerNat;
        const float depth = high == row.top ? 0.f : (row.top - high) * scale;  // bin 0 holds the maximum
        if (depth < (float)(kBins - 1))
            atomicAdd(&sh.hist[(int)depth], 1u);
        uint64_t total = 0;
        if (by_sum && !by_rank) {
            uint64_t v[1] = {sum_whole(slice, c.tid, sh.ring, nullptr, [&](float x) {
                return weight_f(x, row.top, row.filter_r);
            })};
            reduce<1>(c, 2, v);                        // orders the histograms too
            total = v[0];
        } else {
            __syncthreads();
            cl.sync();
        }
        unsigned h[kMaxCluster], count = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            h[r] = r < c.nctas ? cl.map_shared_rank(&sh, r)->hist[c.tid] : 0u;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            count += h[r];
        // The last bin a kept token can be in: the k-th token's; the one where the
        // weights, each taken at its bin's lower edge less a little for rounding, pass
        // top-p's share; min-p's.
        float low = (float)count * __expf(-(float)(c.tid + 1) / kBinsPerNat) * 0.999f;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const unsigned o = __shfl_up_sync(0xffffffffu, count, s);
            const float f = __shfl_up_sync(0xffffffffu, low, s);
            count += c.lane >= s ? o : 0;
            low += c.lane >= s ? f : 0.f;
        }
        if (c.lane == 31) {
            sh.scan[c.warp] = count;
            sh.red[0][c.warp][3] = __float_as_uint(low);
        }
        __syncthreads();
        for (int w = 0; w < c.warp; ++w) {
            count += sh.scan[w];
            low += __uint_as_float((uint32_t)sh.red[0][w][3]);
        }
        bool reach = by_rank ? count >= (unsigned)row.k
                             : by_sum && low >= row.top_p * __ull2float_rn(total) * 9.094947e-13f;   // 2^-40
        // (top-p takes its share of all that top-k kept, min-p or not)
        const float z_min = row.min_p > 0.f && !(by_rank && by_sum) ? -logf(row.min_p) : 1e30f;
        reach = reach || (float)c.tid > z_min * kBinsPerNat + 2.f;
        const int last = __syncthreads_count(!reach);  // bins before the first that reaches
        // ---- the candidates: all logits down to a little below the bin's lower edge ----
        float cut = kNegInf;
        int n = kSearch;
        if (last < kBins - 1) {
            cut = isinf(row.top) ? row.top
                                 : row.top - ((float)last + 1.05f) / scale - fabsf(row.top) * 1e-6f;
            n = gather(c, begin, [&](auto found) {
                if (next >= cut) {                     // in several vectors: read all again
                    each(slice, c.tid, sh.ring, [&](float x, int i) {
                        if (x >= cut)
                            found(x, i);
                    });
                } else if (high >= cut) {
                    float x[Slice<DT>::E];
                    const int one = high_at < slice.head() || high_at >= slice.tail();
#pragma unroll
                    for (int e = 0; e < Slice<DT>::E; ++e)
                        x[e] = e == 0 || !one ? slice.get(high_at + e) : kNegInf;
#pragma unroll
                    for (int e = 0; e < Slice<DT>::E; ++e)
                        if (x[e] >= cut && (e == 0 || !one))
                            found(x[e], high_at + e);
                }
            });
        }
        if (n == kSearch || n > kList) {
            n = select_binned(c, slice, row, cut, total, begin, kept);
            if (n == kSearch)
                kept = select(c, slice, row, total);
        }
        if (n >= 0 && n <= kList) {
            if (c.rank == 0)
                draw_listed(c, row, by_sum, total, n, p, m);
            return;
        }
    }
    float prob;
    const int place = draw(c, slice, row, kept, &prob);
    if (c.tid == 0 && place >= 0) {
        p.token[m] = begin + place;
        if (p.prob)
            p.prob[m] = prob;
    }
}

template <int DT>
cudaError_t launch(const SampleParams& p, int rows, cudaStream_t st)
{
    auto kernel = lbv_sample_kernel<DT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Shared));
    if (e == cudaSuccess && p.ctas > 8)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)p.ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int rows, lbv_dtype dt, cudaStream_t st)
{
    if (dt == LBV_F32)
        return launch<LBV_F32>(p, rows, st);
    return dt == LBV_F16 ? launch<LBV_F16>(p, rows, st) : launch<LBV_BF16>(p, rows, st);
}

}  // namespace lbv

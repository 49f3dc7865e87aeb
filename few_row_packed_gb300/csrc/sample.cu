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
//   1. every thread finds the maximum of its logits, the cluster the row's;
//   2. a bound on how far down the kept tokens can reach.  The thread maxima
//      enter a histogram of (m - l) r in steps of 1/8: the k-th of these few
//      thousand values is at most the row's k-th, and their weights sum to no more
//      than the row's above the same logit, so the first bin that satisfies top-k
//      or top-p on them lies at or below the true cut;
//   3. the few threads whose maximum lies above the bound hand it to the first CTA;
//      those whose next largest does too read their logits again (from L2) and hand
//      over all above it ("candidates").  The other CTAs are done;
//   4. it sorts them by rank; a running sum of their weights gives how many are
//      kept; and sorts these by index, where a running sum gives the token.
// Where the thread maxima do not reach the cut (a large k, a flat row with a
// large top-p), step 2 is tried again with all logits.  Where the candidates do
// not fit the list, tau is found by a search over the bits of the
// (order-preserving) keys, counting and summing above trial values, two bits a
// round, with a cluster barrier in each.  top-p without top-k needs the row's total
// weight: a second pass over the slice.
//
// Nothing of the row stays on chip, so that four CTAs share an SM: while one
// waits at a barrier, the others' loads keep memory busy.
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
constexpr int kMaxCluster = 16;
constexpr float kBinsPerNat = 8.f;
constexpr float kNegInf = -__builtin_huge_valf();

// Vectors of 16 bytes (and their two mask words) on the way to each thread.
struct Ring {
    uint4 v[kAhead][kThreads];
    uint32_t words[kAhead][kThreads][2];
};

struct Shared {
    uint64_t red[2][kWarps][4];            // block reductions, two in flight
    uint64_t all[2][kMaxCluster][4];       // cluster reductions: one slot per CTA
    unsigned hist[kBins];
    uint64_t tops[kMaxCluster];
    uint64_t sums[kWarps];                 // drawn weight of each warp's part
    int counts[kMaxCluster];               // candidates of each CTA
    int found;                             // of this CTA so far
    int listed;                            // of all CTAs so far (in the first)
    unsigned scan[kWarps];
    int pick;                              // place of the drawn token
    float pick_prob;
    uint64_t list[kList];                  // candidates: key, then the index's complement
    union {
        Ring ring;                         // of the passes over the slice
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
// maximum weighs exactly 1 (the maximum may be +inf), a masked one 0.
__device__ __forceinline__ float weight_f(float x, float top, float r)
{
    const float z = x == top ? 0.f : __fmul_rn(__fsub_rn(x, top), r);
    return x == kNegInf ? 0.f : expf(z);
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
    int tid, warp, lane, rank, nctas, round;
};

// Sums N values over the CTA's threads, or (wide) the cluster's; every thread
// gets the result.  below[] (optional): the sums over the CTAs of lower rank.
template <int N>
__device__ __noinline__ void reduce(Ctx& c, bool wide, uint64_t (&v)[N], uint64_t* below = nullptr)
{
    Shared& sh = *c.sh;
    const int b = c.round++ & 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = shfl_add(v[i]);
        if (c.lane == 0)
            sh.red[b][c.warp][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            v[i] += sh.red[b][w][i];
    }
    if (wide) {
        cg::cluster_group cl = cg::this_cluster();
        if (c.tid < c.nctas) {
            Shared* to = cl.map_shared_rank(c.sh, c.tid);
#pragma unroll
            for (int i = 0; i < N; ++i)
                to->all[b][c.rank][i] = v[i];
        }
        cl.sync();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint64_t t = 0, lo = 0;
            for (int r = 0; r < c.nctas; ++r) {
                lo = r == c.rank ? t : lo;
                t += sh.all[b][r][i];
            }
            v[i] = t;
            if (below)
                below[i] = lo;
        }
    } else if (below) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            below[i] = 0;
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
    const unsigned char* row;              // its first element
    const uint32_t* words;                 // its mask words, or NULL
    int n;
    // a logit as the search sees it; `allowed`: its mask bit
    static __device__ __forceinline__ float clean(float v, bool allowed)
    {
        v = __fadd_rn(v, 0.f);
        return v != v || !allowed ? kNegInf : v;
    }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t b = SIZE == 4 ? __ldg(reinterpret_cast<const uint32_t*>(row) + i)
                                     : __ldg(reinterpret_cast<const uint16_t*>(row) + i);
        return clean(to_f32<DT>(b), !words || ((__ldg(words + (i >> 5)) >> (i & 31)) & 1u));
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

// Calls f(value, index) for the thread's logits of the slice, indexes ascending:
// 16-byte copies between the first and the last aligned address, several of them
// in flight, into places of the ring that only this thread reads (in registers, a
// rotation of the buffers would wait for the copy that was just asked for).
// AT_ONCE elements of a vector are unrolled.
template <int AT_ONCE, int DT, typename F>
__device__ __forceinline__ void each(const Slice<DT>& s, int tid, Ring& ring, F f)
{
    constexpr int SIZE = Slice<DT>::SIZE, E = 16 / SIZE;
    const uintptr_t a = reinterpret_cast<uintptr_t>(s.row);
    const int head = min(s.n, (int)(((16 - (a & 15)) & 15) / SIZE));
    const int body = (s.n - head) / E, tail = head + body * E;
    const uint4* v = reinterpret_cast<const uint4*>(a + head * SIZE);
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
        f(s.get(tid), tid);
    int st = 0;
#pragma unroll 1
    for (int i = tid; i < body; i += kThreads) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead - 1) : "memory");
        const uint4 w = ring.v[st][tid];
        const int d = head + i * E;
        const uint32_t m =
            s.words ? __funnelshift_r(ring.words[st][tid][0], ring.words[st][tid][1], d & 31) : ~0u;
        ask(i + kAhead * kThreads, st);
        st = st + 1 == kAhead ? 0 : st + 1;
        const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += AT_ONCE)
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                const int e = e0 + k;
                uint32_t b;
                if constexpr (DT == LBV_F32) {
                    b = AT_ONCE == 4 ? q[k] : e < 2 ? (e & 1 ? q[1] : q[0]) : (e & 1 ? q[3] : q[2]);
                } else {
                    const uint32_t r = AT_ONCE == 8 ? q[k / 2] : e < 4 ? (e < 2 ? q[0] : q[1]) : (e < 6 ? q[2] : q[3]);
                    b = e & 1 ? r >> 16 : r & 0xFFFFu;
                }
                f(s.clean(to_f32<DT>(b), (m >> e) & 1u), d + e);
            }
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    if (tail + tid < s.n)                  // fewer than E of them
        f(s.get(tail + tid), tail + tid);
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
__device__ __forceinline__ uint32_t search(Ctx& c, const D& d, F f, Test test)
{
    uint32_t t = 0;
    for (int bit = 30; bit >= 0; bit -= 2) {
        uint64_t s1 = 0, s2 = 0, s3 = 0;
        const uint32_t t1 = t | (1u << bit), t2 = t | (2u << bit), t3 = t | (3u << bit);
        each<2>(d, c.tid, c.sh->ring, [&](float x, int) {
            const uint32_t k = key_of(x);
            if (k >= t1) {
                const uint64_t w = f(x);
                s1 += w;
                s2 += k >= t2 ? w : 0;
                s3 += k >= t3 ? w : 0;
            }
        });
        uint64_t v[3] = {s1, s2, s3};
        reduce<3>(c, true, v);
        t = test(t3, v[2]) ? t3 : test(t2, v[1]) ? t2 : test(t1, v[0]) ? t1 : t;
    }
    return t;
}

// tau and its ties by search.  total: the weight of the whole row (without top-k).
template <typename D>
__device__ __noinline__ Kept select(Ctx& c, const D& d, const Row& row, uint64_t total)
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
        each<2>(d, c.tid, c.sh->ring, [&](float x, int) {
            if (key_of(x) > tau_k) {
                n += 1;
                sum += weight(x);
            }
        });
        uint64_t v[2] = {n, sum};
        reduce<2>(c, true, v);
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
        each<2>(d, c.tid, c.sh->ring, [&](float x, int) { sum += key_of(x) > tau ? weight(x) : 0; });
        uint64_t v[1] = {sum};
        reduce<1>(c, true, v);
        const uint64_t w = weight(of_key(tau));
        const uint64_t j = w ? (limit - v[0] + w - 1) / w : 1;
        kept.ties = tau == tau_k && j > kept.ties ? kept.ties : j;
        kept.tau = tau;
    }
    return kept;
}

// Draws from the kept tokens of the domain in index order.  Returns the place
// in the domain, or -1 where another CTA's slice holds it; *prob its
// probability among the kept ones.
template <typename D>
__device__ __noinline__ int draw(Ctx& c, const D& d, const Row& row, const Kept& kept, float* prob)
{
    Shared& sh = *c.sh;
    const int groups = (d.n + 31) / 32, per = (groups + kWarps - 1) / kWarps;
    const int g0 = min(c.warp * per, groups), g1 = min(g0 + per, groups);
    const unsigned before = (1u << c.lane) - 1;
    // ties in index order ahead of this warp
    uint64_t tie_base = 0;
    if (kept.ties != ~0ull) {
        unsigned mine = 0;
        for (int g = g0; g < g1; ++g) {
            const int i = g * 32 + c.lane;
            mine += i < d.n && key_of(d.get(i)) == kept.tau;
        }
        mine = __reduce_add_sync(0xffffffffu, mine);
        __syncthreads();
        if (c.lane == 0)
            sh.scan[c.warp] = mine;
        uint64_t v[1] = {c.lane == 0 ? mine : 0u}, lo[1];
        reduce<1>(c, true, v, lo);      // its barrier orders the scan array
        tie_base = lo[0];
        for (int w = 0; w < c.warp; ++w)
            tie_base += sh.scan[w];
    }
    // visits the warp's tokens in index order: f(place, weight) by all lanes
    auto visit = [&](auto f) {
        uint64_t ties = tie_base;
#pragma unroll 4
        for (int g = g0; g < g1; ++g) {
            const int i = g * 32 + c.lane;
            const float x = i < d.n ? d.get(i) : kNegInf;
            const uint32_t k = key_of(x);
            const bool tie = i < d.n && k == kept.tau;
            const unsigned tied = __ballot_sync(0xffffffffu, tie);
            const bool in = i < d.n && (k > kept.tau || (tie && ties + __popc(tied & before) < kept.ties));
            ties += __popc(tied);
            uint64_t w = 0;
            if (in && weight_f(x, row.top, row.filter_r) >= row.min_p)
                w = whole(weight_f(x, row.top, row.draw_r));
            if (f(i, w))
                return;
        }
    };
    uint64_t sum = 0;
    visit([&](int, uint64_t w) { sum += w; return false; });
    sum = shfl_add(sum);
    __syncthreads();
    if (c.lane == 0)
        sh.sums[c.warp] = sum;
    if (c.tid == 0)
        sh.pick = -1;
    uint64_t v[1] = {c.lane == 0 ? sum : 0}, lo[1];
    reduce<1>(c, true, v, lo);
    const uint64_t total = v[0];
    uint64_t at = lo[0];
    for (int w = 0; w < c.warp; ++w)
        at += sh.sums[w];
    uint32_t f = fraction24(row.u);
    f = f > 16777215u ? 16777215u : f;
    const uint64_t target = part(f, total);
    if (target >= at && target < at + sum) {
        visit([&](int i, uint64_t w) {
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

// The block's sum of v, and in `before` that of the threads before this one.
__device__ __noinline__ uint64_t block_scan(Ctx& c, uint64_t v, uint64_t& before)
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

// Draws from the n candidates of the list, of which every kept token is one.
// total: the weight of the whole row (without top-k).
__device__ __forceinline__ void draw_listed(Ctx& c, const Row& row, bool by_sum, uint64_t total, int n,
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
    c.round = 0;
    const int m = blockIdx.x / p.ctas;
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
    float high = kNegInf, next = kNegInf;              // the largest logit, the next one
    int high_at = 0;
    each<DT == LBV_F32 ? 4 : 8>(slice, c.tid, sh.ring, [&](float v, int i) {
        next = fmaxf(next, fminf(v, high));
        high_at = v > high ? i : high_at;
        high = fmaxf(high, v);
    });
    sh.hist[c.tid] = 0;
    if (c.tid == 0)
        sh.found = sh.listed = 0;
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
        if (c.rank == 0 && c.tid == 0) {
            const bool none = best == 0 || row.top == kNegInf;
            p.token[m] = none ? -1 : first;
            if (p.prob)
                p.prob[m] = none ? 0.f : 1.f;
        }
        return;
    }

    Kept kept = {0u, ~0ull};
    const bool by_rank = row.k > 0 && row.k < p.N, by_sum = row.top_p < 1.f;
    row.k = by_rank ? row.k : 0;
    uint64_t total = 0;
    if (by_rank || by_sum) {
        const float scale = row.filter_r * kBinsPerNat;
        auto bin_of = [&](float v) {                   // bin 0 holds the maximum
            const float b = v == row.top ? 0.f : (row.top - v) * scale;
            return b < (float)(kBins - 1) ? (int)b : kBins - 1;
        };
        Shared* to = cl.map_shared_rank(&sh, 0);
        for (int all = 0; all < 2; ++all) {
            // ---- the histogram, and with it (once) the row's weight ----
            if (all == 0) {
                const int b = bin_of(high);
                if (b < kBins - 1)
                    atomicAdd(&sh.hist[b], 1u);
                if (by_rank) {
                    __syncthreads();
                    cl.sync();
                } else {
                    uint64_t sum = 0;
                    each<DT == LBV_F32 ? 4 : 8>(slice, c.tid, sh.ring, [&](float x, int) {
                        sum += whole(weight_f(x, row.top, row.filter_r));
                    });
                    uint64_t v[1] = {sum};
                    reduce<1>(c, true, v);             // orders the histograms too
                    total = v[0];
                }
            } else {
                cl.sync();                             // the first one has been read
                sh.hist[c.tid] = 0;
                if (c.tid == 0)
                    sh.found = sh.listed = 0;
                __syncthreads();
                each<2>(slice, c.tid, sh.ring, [&](float x, int) {
                    const int b = bin_of(x);
                    if (b < kBins - 1)
                        atomicAdd(&sh.hist[b], 1u);
                });
                cl.sync();
            }
            unsigned h[kMaxCluster], here = 0;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                h[r] = r < c.nctas ? cl.map_shared_rank(&sh, r)->hist[c.tid] : 0u;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                here += h[r];
            // The last bin a kept token can be in: the k-th token's; the one
            // where the weights, each taken at its bin's lower edge less a little
            // for rounding, pass top-p's share; min-p's.
            unsigned count = here;
            float low = (float)here * __expf(-(float)(c.tid + 1) / kBinsPerNat) * 0.999f;
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
                                 : low >= row.top_p * __ull2float_rn(total) * 9.094947e-13f;   // 2^-40
            // (top-p takes its share of all that top-k kept, min-p or not)
            const float z_min = row.min_p > 0.f && !(by_rank && by_sum) ? -logf(row.min_p) : 1e30f;
            reach = reach || (float)c.tid > z_min * kBinsPerNat + 2.f;
            const int last = __syncthreads_count(!reach);      // bins before the first that reaches
            if (last >= kBins - 1)
                continue;
            // ---- the candidates: all logits down to a little below the bin's lower edge ----
            const float cut = isinf(row.top) ? row.top
                                             : row.top - ((float)last + 1.05f) / scale - fabsf(row.top) * 1e-6f;
            auto found = [&](float x, int i) {
                if (x >= cut) {
                    atomicAdd(&sh.found, 1);
                    const int at = atomicAdd(&to->listed, 1);
                    if (at < kList)
                        to->list[at] = ((uint64_t)key_of(x) << 32) | (0xFFFFFFFFu - (uint32_t)(begin + i));
                }
            };
            if (next >= cut)
                each<2>(slice, c.tid, sh.ring, found);          // more than one: read them again
            else
                found(high, high_at);
            __syncthreads();
            if (c.tid < c.nctas)
                cl.map_shared_rank(&sh, c.tid)->counts[c.rank] = sh.found;
            cl.sync();
            int n = 0;
            for (int r = 0; r < c.nctas; ++r)
                n += sh.counts[r];
            if (n <= kList) {
                if (c.rank == 0)
                    draw_listed(c, row, by_sum, total, n, p, m);
                return;
            }
            // (the thread maxima's bound was too low: all logits give a closer one)
        }
        kept = select(c, slice, row, total);
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
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)p.ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
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

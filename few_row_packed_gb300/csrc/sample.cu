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
// A row takes one thread-block cluster whose CTAs stage disjoint slices of it
// in shared memory, so the logits are read from memory once (the bound of a
// large batch); everything after the first pass works on chip.  Selecting
// needs no sort of the row:
//   1. the row's maximum (a cluster barrier);
//   2. a bound on how far down the kept tokens can reach.  Each thread's own
//      maximum enters a histogram of (m - l) r in steps of 1/16 (a barrier): the
//      k-th of these few thousand values is at most the row's k-th, and their
//      weights sum to no more than the row's above the same logit, so the first
//      bin that satisfies top-k or top-p on them lies at or below the true cut;
//   3. the tokens above that bound, a few more than are kept, go in index order
//      to the first CTA (a barrier), and the other CTAs are done;
//   4. each of these candidates counts and sums those ranked before it, which
//      decides whether it is kept, and an index-order running sum gives the
//      token.  Up to kRanked candidates; a longer list finds tau by a search
//      over the bits of the (order-preserving) keys, counting and summing above
//      trial values, two bits a round.
// Where the thread maxima do not reach the cut (a large k, a flat row with a
// large top-p), step 2 is tried again with all logits, and where the candidates
// do not fit the list, the search runs over the slices of all CTAs, with a
// cluster barrier in each round.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "step_internal.h"

namespace lbv {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;            // one thread per bin
constexpr int kList = 4096;                // candidates the first CTA can take
constexpr int kRanked = 384;               // candidates ranked by pairs
constexpr int kMaxCluster = 16;
constexpr float kBinsPerNat = 16.f;
constexpr float kNegInf = -__builtin_huge_valf();

struct Shared {
    uint64_t red[2][kWarps][4];            // block reductions, two in flight
    uint64_t all[2][kMaxCluster][4];       // cluster reductions: one slot per CTA
    unsigned hist[kBins];
    uint64_t tops[kMaxCluster];
    uint64_t sums[kWarps];                 // drawn weight of each warp's part
    int counts[kMaxCluster];               // candidates of each CTA
    unsigned scan[kWarps];
    int pick;                              // place of the drawn token
    float pick_prob;
    uint4 pairs[kRanked];                  // key and weight of the ranked candidates
    float list_x[kList];                   // a segment for each CTA
    int list_i[kList];
};

// Order-preserving key of a logit (-0 made +0 before); -inf has a key above 0.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// exp((x - top) r) in fp32, every operation rounded once; a token at the
// maximum weighs exactly 1 (the maximum may be +inf), a masked one 0.
__device__ __forceinline__ float weight_f(float x, float top, float r)
{
    const float z = x == top ? 0.f : __fmul_rn(__fsub_rn(x, top), r);
    return x == kNegInf ? 0.f : expf(z);
}

__device__ __forceinline__ uint64_t whole(float w)
{
    return (uint64_t)__fmul_rn(fmaxf(w, 0.f), 1099511627776.f);   // 2^40, truncated; NaN gives 0
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

// The tokens a search runs over: a CTA's slice of the row, cluster-wide, or
// the candidate list of the first CTA alone.
struct Domain {
    const float* x;
    int n;
    bool wide;
};

struct Ctx {
    Shared* sh;
    int tid, warp, lane, rank, nctas, round;
};

// Sums N values over the domain's threads; every thread gets the result.
// below[] (optional): the sums over the CTAs of lower rank.
template <int N>
__device__ __forceinline__ void reduce(Ctx& c, bool wide, uint64_t (&v)[N], uint64_t* below = nullptr)
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
        uint64_t t = c.lane < kWarps ? sh.red[b][c.lane][i] : 0;
        v[i] = shfl_add(t);
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

// The largest key t for which test(sums of f over the tokens with key >= t)
// holds; it holds at 0.  f(x) is a count or a weight, test is monotone in t.
template <typename F, typename Test>
__device__ __forceinline__ uint32_t search(Ctx& c, const Domain& d, F f, Test test)
{
    uint32_t t = 0;
    for (int bit = 30; bit >= 0; bit -= 2) {
        uint64_t v[3] = {0, 0, 0};
        const uint32_t t1 = t | (1u << bit), t2 = t | (2u << bit), t3 = t | (3u << bit);
        for (int i = c.tid; i < d.n; i += kThreads) {
            const uint32_t k = key_of(d.x[i]);
            if (k >= t1) {
                const uint64_t w = f(d.x[i]);
                v[0] += w;
                v[1] += k >= t2 ? w : 0;
                v[2] += k >= t3 ? w : 0;
            }
        }
        reduce<3>(c, d.wide, v);
        t = test(t3, v[2]) ? t3 : test(t2, v[1]) ? t2 : test(t1, v[0]) ? t1 : t;
    }
    return t;
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

__device__ Kept select(Ctx& c, const Domain& d, const Row& row, bool have_total, uint64_t total)
{
    Kept kept = {0u, ~0ull};
    uint32_t tau_k = 0;
    if (row.k > 0) {
        const uint64_t k = (uint64_t)row.k;
        tau_k = search(c, d, [](float) { return (uint64_t)1; },
                       [&](uint32_t, uint64_t n) { return n >= k; });
        // its ties, and what lies above
        uint64_t v[2] = {0, 0};
        for (int i = c.tid; i < d.n; i += kThreads)
            if (key_of(d.x[i]) > tau_k) {
                v[0] += 1;
                v[1] += whole(weight_f(d.x[i], row.top, row.filter_r));
            }
        reduce<2>(c, d.wide, v);
        kept.tau = tau_k;
        kept.ties = k - v[0];
        // fewer than k tokens may be left above a masked one: its weight is 0
        const uint32_t b = tau_k ^ (tau_k & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu);
        total = v[1] + kept.ties * whole(weight_f(__uint_as_float(b), row.top, row.filter_r));
    } else if (!have_total) {
        uint64_t v[1] = {0};
        for (int i = c.tid; i < d.n; i += kThreads)
            v[0] += whole(weight_f(d.x[i], row.top, row.filter_r));
        reduce<1>(c, d.wide, v);
        total = v[0];
    }
    if (row.top_p < 1.f) {
        const uint64_t limit = part(fraction24(row.top_p), total);
        if (limit == 0)
            return Kept{key_of(row.top), 1};
        auto weight = [&](float x) { return whole(weight_f(x, row.top, row.filter_r)); };
        const uint32_t tau = search(c, d, weight, [&](uint32_t t, uint64_t s) {
            return t <= tau_k || s >= limit;
        });
        uint64_t v[1] = {0};
        for (int i = c.tid; i < d.n; i += kThreads)
            if (key_of(d.x[i]) > tau)
                v[0] += weight(d.x[i]);
        reduce<1>(c, d.wide, v);
        const uint32_t b = tau ^ (tau & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu);
        const uint64_t w = weight(__uint_as_float(b));
        const uint64_t j = w ? (limit - v[0] + w - 1) / w : 1;
        kept.ties = tau == tau_k && j > kept.ties ? kept.ties : j;
        kept.tau = tau;
    }
    return kept;
}

// Draws from the kept tokens of the domain in index order.  Returns the place
// in the domain, or -1 where another CTA's slice holds it; *prob its
// probability among the kept ones.
__device__ int draw(Ctx& c, const Domain& d, const Row& row, const Kept& kept, float* prob)
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
            mine += i < d.n && key_of(d.x[i]) == kept.tau;
        }
        mine = __reduce_add_sync(0xffffffffu, mine);
        __syncthreads();
        if (c.lane == 0)
            sh.scan[c.warp] = mine;
        uint64_t v[1] = {c.lane == 0 ? mine : 0u}, lo[1];
        reduce<1>(c, d.wide, v, lo);       // its barrier orders the scan array
        tie_base = lo[0];
        for (int w = 0; w < c.warp; ++w)
            tie_base += sh.scan[w];
    }
    // visits the warp's tokens in index order: f(place, weight) by all lanes
    auto visit = [&](auto f) {
        uint64_t ties = tie_base;
        for (int g = g0; g < g1; ++g) {
            const int i = g * 32 + c.lane;
            const float x = i < d.n ? d.x[i] : kNegInf;
            const uint32_t k = key_of(x);
            const bool tie = i < d.n && k == kept.tau;
            const unsigned tied = __ballot_sync(0xffffffffu, tie);
            bool in = i < d.n && (k > kept.tau || (tie && ties + __popc(tied & before) < kept.ties));
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
    reduce<1>(c, d.wide, v, lo);
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
                *prob = __fdiv_rn(__ull2float_rn(w), __ull2float_rn(total));
                sh.pick_prob = *prob;
            }
            return true;
        });
    }
    __syncthreads();
    *prob = sh.pick_prob;
    return sh.pick;
}

// Writes the slice's tokens of logit >= cut in index order to to_x, to_i (`cap`
// of them at most) and returns how many there are.
__device__ int collect(Ctx& c, const float* x, int n, float cut, int begin, int cap, float* to_x,
                       int* to_i)
{
    Shared& sh = *c.sh;
    // 128 logits a step: four neighbours a lane
    const int steps = (n + 127) / 128, per = (steps + kWarps - 1) / kWarps;
    const int g0 = min(c.warp * per, steps), g1 = min(g0 + per, steps);
    const unsigned before = (1u << c.lane) - 1;
    auto hits = [&](int g, float (&v)[4], unsigned (&b)[4]) {
        const int i = g * 128 + c.lane * 4;
        if (i + 3 < n) {
            const float4 q = *reinterpret_cast<const float4*>(x + i);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = i + e < n ? x[i + e] : kNegInf;
        }
        const bool any = (v[0] >= cut && i < n) || (v[1] >= cut && i + 1 < n) ||
                         (v[2] >= cut && i + 2 < n) || (v[3] >= cut && i + 3 < n);
        if (!__any_sync(0xffffffffu, any))
            return 0;
        int k = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            b[e] = __ballot_sync(0xffffffffu, v[e] >= cut && i + e < n);
            k += __popc(b[e]);
        }
        return k;
    };
    float v[4];
    unsigned b[4];
    unsigned found = 0;
    for (int g = g0; g < g1; ++g)
        found += hits(g, v, b);
    if (c.lane == 0)
        sh.scan[c.warp] = found;
    __syncthreads();
    int at = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        at += w < c.warp ? sh.scan[w] : 0;
        all += sh.scan[w];
    }
    if (all <= cap && found)
        for (int g = g0; g < g1; ++g) {
            const int k = hits(g, v, b);
            if (!k)
                continue;
            int to = at + __popc(b[0] & before) + __popc(b[1] & before) + __popc(b[2] & before) +
                     __popc(b[3] & before);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((b[e] >> c.lane) & 1u) {
                    to_x[to] = v[e];
                    to_i[to] = begin + g * 128 + c.lane * 4 + e;
                    ++to;
                }
            at += k;
        }
    return all;
}

// Draws from n <= kRanked candidates in index order, one a thread (list place
// `at`, -1: none): what is ranked before a candidate decides whether it is kept.
__device__ void rank_and_draw(Ctx& c, const Row& row, bool by_sum, uint64_t total, int n, int at,
                              const SampleParams& p, int m)
{
    Shared& sh = *c.sh;
    const bool in = c.tid < n;
    const float x = in ? sh.list_x[at] : kNegInf;
    const int index = in ? sh.list_i[at] : 0;
    const uint32_t key = key_of(x);
    const float wf = weight_f(x, row.top, row.filter_r);
    const uint64_t w = in ? whole(wf) : 0;
    if (in)
        sh.pairs[c.tid] = make_uint4(key, (uint32_t)w, (uint32_t)(w >> 32), 0u);
    __syncthreads();
    unsigned rank = 0;
    uint64_t ahead = 0;
    if (c.warp * 32 < n) {
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const uint4 o = sh.pairs[j];
            if (o.x > key || (o.x == key && j < c.tid)) {
                ++rank;
                ahead += ((uint64_t)o.z << 32) | o.y;
            }
        }
    }
    const bool by_rank = row.k > 0;
    bool keep = in && (!by_rank || rank < (unsigned)row.k);
    if (by_sum) {
        if (by_rank) {
            uint64_t v[1] = {keep ? w : 0};
            reduce<1>(c, false, v);
            total = v[0];
        }
        keep = keep && (rank == 0 || ahead < part(fraction24(row.top_p), total));
    }
    keep = keep && wf >= row.min_p;
    const uint64_t dw = keep ? whole(weight_f(x, row.top, row.draw_r)) : 0;
    uint64_t upto = dw;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, upto, s);
        upto += c.lane >= s ? o : 0;
    }
    if (c.lane == 31)
        sh.sums[c.warp] = upto;
    __syncthreads();
    uint64_t all = 0, below = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        below = i == c.warp ? all : below;
        all += sh.sums[i];
    }
    upto += below;
    uint32_t f = fraction24(row.u);
    f = f > 16777215u ? 16777215u : f;
    const uint64_t target = part(f, all);
    if (upto > target && upto - dw <= target) {
        p.token[m] = index;
        if (p.prob)
            p.prob[m] = __fdiv_rn(__ull2float_rn(dw), __ull2float_rn(all));
    }
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i)
{
    if constexpr (DT == LBV_F32)
        return static_cast<const float*>(p)[i];
    else if constexpr (DT == LBV_F16)
        return __half2float(__ushort_as_half(static_cast<const uint16_t*>(p)[i]));
    else
        return __bfloat162float(__ushort_as_bfloat16(static_cast<const uint16_t*>(p)[i]));
}

// The thread's largest logit so far and its index in the slice (the first of
// equal ones, as the thread's indices ascend).
struct Best {
    float x = kNegInf;
    int i = -1;
};

// Copies n logits from element `at` on into shared memory as fp32, masked ones
// and NaN as -inf, and finds the thread's maximum: 16-byte loads between the
// first and the last aligned address.
template <int DT>
__device__ __forceinline__ Best stage(const void* src, int64_t at, int n, const uint32_t* words,
                                      float* x, int tid)
{
    constexpr int E = DT == LBV_F32 ? 4 : 8;           // elements of 16 bytes
    constexpr int SIZE = 16 / E;
    Best best;
    auto put = [&](int i, float v) {
        v = __fadd_rn(v, 0.f);                         // -0 becomes +0
        const bool out = v != v || (words && !((words[i >> 5] >> (i & 31)) & 1u));
        v = out ? kNegInf : v;
        x[i] = v;
        if (v > best.x) {
            best.x = v;
            best.i = i;
        }
    };
    const uintptr_t a = reinterpret_cast<uintptr_t>(src) + (uintptr_t)at * SIZE;
    const int head = min(n, (int)(((16 - (a & 15)) & 15) / SIZE));
    const int body = (n - head) / E;
    if (tid < head)
        put(tid, load1<DT>(src, at + tid));
    const uint4* v = reinterpret_cast<const uint4*>(a + head * SIZE);
    constexpr int U = 8;
    for (int i = tid; i < body; i += U * kThreads) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kThreads < body)
                w[u] = __ldcs(v + i + u * kThreads);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u * kThreads < body) {
                const int d = head + (i + u * kThreads) * E;
                const uint32_t q[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (DT == LBV_F32) {
                        put(d + e, __uint_as_float(q[e]));
                    } else if constexpr (DT == LBV_F16) {
                        put(d + 2 * e, __half2float(__ushort_as_half((uint16_t)q[e])));
                        put(d + 2 * e + 1, __half2float(__ushort_as_half((uint16_t)(q[e] >> 16))));
                    } else {
                        put(d + 2 * e, __uint_as_float(q[e] << 16));
                        put(d + 2 * e + 1, __uint_as_float(q[e] & 0xFFFF0000u));
                    }
                }
            }
    }
    for (int i = head + body * E + tid; i < n; i += kThreads)
        put(i, load1<DT>(src, at + i));
    return best;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) lbv_sample_kernel(const __grid_constant__ SampleParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    float* x = reinterpret_cast<float*>(smem + sizeof(Shared));
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
    const int n = min(p.slice, p.N - begin);

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

    // ---- the slice, masked, and the row's first maximum ----
    sh.hist[c.tid] = 0;
    const Best mine = stage<DT>(p.logits, (int64_t)m * p.ld + begin, n,
                                p.mask ? p.mask + (int64_t)m * p.mask_ld + begin / 32 : nullptr, x, c.tid);
    uint64_t best = 0;
    if (n > 0)       // a row of -inf has a key above 0 too
        best = ((uint64_t)key_of(mine.x) << 32) | (0xFFFFFFFFu - (uint32_t)(begin + mine.i));
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
        for (int w = 0; w < kWarps; ++w)
            b = sh.red[0][w][0] > b ? sh.red[0][w][0] : b;
        cl.map_shared_rank(&sh, c.tid)->tops[c.rank] = b;
    }
    cl.sync();
    best = 0;
    for (int r = 0; r < c.nctas; ++r)
        best = sh.tops[r] > best ? sh.tops[r] : best;
    const uint32_t kb = (uint32_t)(best >> 32);
    row.top = __uint_as_float(kb ^ (kb & 0x80000000u ? 0x80000000u : 0xFFFFFFFFu));
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

    Domain d = {x, n, true};
    Kept kept = {0u, ~0ull};
    const bool by_rank = row.k > 0 && row.k < p.N, by_sum = row.top_p < 1.f;
    row.k = by_rank ? row.k : 0;
    if (by_rank || by_sum) {
        const float scale = row.filter_r * kBinsPerNat;
        auto bin_of = [&](float v) {                   // bin 0 holds the maximum
            const float b = v == row.top ? 0.f : (row.top - v) * scale;
            return b < (float)(kBins - 1) ? (int)b : kBins - 1;
        };
        uint64_t v[1] = {0}, total = 0;
        bool listed = false;
        for (int all = 0; all < 2 && !listed; ++all) {
            // ---- the histogram, and with it (once) the row's weight ----
            if (all == 0) {
                const int b = bin_of(mine.x);
                if (b < kBins - 1)
                    atomicAdd(&sh.hist[b], 1u);
                if (!by_rank)
                    for (int i = c.tid; i < n; i += kThreads)
                        v[0] += whole(weight_f(x[i], row.top, row.filter_r));
                reduce<1>(c, true, v);                 // orders the histograms too
                total = v[0];
            } else {
                cl.sync();                             // the first one has been read
                sh.hist[c.tid] = 0;
                __syncthreads();
                for (int i = c.tid; i < n; i += kThreads) {
                    const int b = bin_of(x[i]);
                    if (b < kBins - 1)
                        atomicAdd(&sh.hist[b], 1u);
                }
                cl.sync();
            }
            unsigned h[kMaxCluster];
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r)
                h[r] = r < c.nctas ? cl.map_shared_rank(&sh, r)->hist[c.tid] : 0u;
            unsigned here = 0;
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
            const int cap = kList / c.nctas;
            Shared* to = cl.map_shared_rank(&sh, 0);
            const int found = collect(c, x, n, cut, begin, cap, to->list_x + c.rank * cap,
                                      to->list_i + c.rank * cap);
            if (c.tid < c.nctas)
                cl.map_shared_rank(&sh, c.tid)->counts[c.rank] = found;
            cl.sync();
            listed = true;
            for (int r = 0; r < c.nctas; ++r)
                listed = listed && sh.counts[r] <= cap;
        }
        if (listed) {
            if (c.rank != 0)
                return;
            const int cap = kList / c.nctas;
            int before = 0, mine_at = -1;   // thread t < kRanked takes candidate t
            for (int r = 0; r < c.nctas; ++r) {
                const int f = sh.counts[r];
                if (c.tid >= before && c.tid < before + f)
                    mine_at = r * cap + c.tid - before;
                before += f;
            }
            if (before <= kRanked) {
                rank_and_draw(c, row, by_sum, total, before, mine_at, p, m);
                return;
            }
            // the list moves to the start of the slice, which is done with
            before = 0;
            for (int r = 0; r < c.nctas; ++r) {
                const int f = sh.counts[r];
                for (int i = c.tid; i < f; i += kThreads)
                    x[before + i] = sh.list_x[r * cap + i];
                before += f;
            }
            __syncthreads();
            d = Domain{x, before, false};
        }
        kept = select(c, d, row, true, total);
    }
    float prob = 0.f;
    const int place = draw(c, d, row, kept, &prob);
    if (place >= 0 && c.tid == 0) {
        int at = begin + place;
        if (!d.wide) {                                 // the list's segments, in CTA order
            int r = 0, i = place;
            while (i >= sh.counts[r])
                i -= sh.counts[r++];
            at = sh.list_i[r * (kList / c.nctas) + i];
        }
        p.token[m] = at;
        if (p.prob)
            p.prob[m] = prob;
    }
}

template <int DT>
cudaError_t launch(const SampleParams& p, int rows, cudaStream_t st)
{
    const size_t smem = sizeof(Shared) + (size_t)(p.slice > kList ? p.slice : kList) * 4;
    auto kernel = lbv_sample_kernel<DT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxSampleSmem);
    if (e == cudaSuccess && p.ctas > 8)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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

// Slices of at most this many logits leave room for the rest (see Shared).
int sample_max_slice()
{
    return (int)((kMaxSampleSmem - sizeof(Shared)) / 4 / 32 * 32);
}

cudaError_t launch_sample(const SampleParams& p, int rows, lbv_dtype dt, cudaStream_t st)
{
    if (dt == LBV_F32)
        return launch<LBV_F32>(p, rows, st);
    return dt == LBV_F16 ? launch<LBV_F16>(p, rows, st) : launch<LBV_BF16>(p, rows, st);
}

}  // namespace lbv

// attend_common.cuh -- what the two attention kernels share: PTX wrappers,
// the geometry of a request's keys and the copies of key blocks out of the
// paged cache.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend_internal.h"

namespace lbv {
namespace att {

__device__ __forceinline__ uint32_t smem_u32(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait (`limit` SM clocks): false if it gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, unsigned limit)
{
    if (mbar_try(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity))
        if (clock64() - t0 > (long long)limit)
            return false;
    return true;
}

__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

__device__ __forceinline__ void named_bar_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// One box of a cache tensor map: 64 elements of a head from element x on, the
// map's rows of `page` from `slot` on (x is 0 or 64; a page outside the cache
// fills zeros).
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int slot,
                                        int head, int page, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst), "l"(map), "r"(x), "r"(slot),
        "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p)
{
    asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p) : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (DT == LBV_F16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The two values as they were rounded.
template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t r)
{
    if constexpr (DT == LBV_F16)
        return __half22float2(reinterpret_cast<const __half2&>(r));
    else
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
}

// Whether a copy of keys [key, key + n) is of use to a tile that sees [lo, hi) and the sinks.
__device__ __forceinline__ bool wanted(const AttendParams& p, int lo, int hi, int key, int n)
{
    return key < hi && (key + n > lo || key < p.sinks);
}

// A request's share of the batch.
struct Request {
    int q0, n;             // first row, new tokens
    int kv;                // context length, new tokens included
    int first;             // cache position of new token 0 (may be negative)
    int keys;              // keys that exist: kv, at most what the block table maps
};

__device__ __forceinline__ Request request_of(const AttendParams& p, int r)
{
    Request q;
    q.q0 = p.batch.q_start[r];
    // rows past `tokens` do not exist, whatever q_start says
    q.n = max(0, min(p.batch.q_start[r + 1], p.batch.tokens) - q.q0);
    q.kv = p.batch.kv_len[r];
    q.first = q.kv - (p.batch.q_start[r + 1] - q.q0);
    q.keys = max(0, (int)min((int64_t)q.kv, (int64_t)p.batch.table_pages << p.kv.page_shift));
    return q;
}

// Keys [lo, hi) that new tokens i0..i1 of a request can see, beside the sinks.
__device__ __forceinline__ void key_range(const AttendParams& p, const Request& q, int i0, int i1,
                                          int& lo, int& hi)
{
    hi = p.tree ? q.keys : max(0, min(q.keys, q.first + i1 + 1));
    lo = p.window > 0 ? max(0, q.first + i0 - p.window + 1) : 0;
}

// Whether new token i at position pos (tree word w) sees `key`.
__device__ __forceinline__ bool sees(const AttendParams& p, const Request& q, int pos, uint64_t w,
                                     int key)
{
    bool s;
    if (p.tree) {
        const int j = key - q.first;
        s = j < 0 || (j < 64 && ((w >> j) & 1));
    } else {
        s = key <= pos;
    }
    return s && key < q.keys && (p.window <= 0 || key > pos - p.window || key < p.sinks);
}

// The same for 32 keys from key0 on, as bits; `first` and `keys` of the request.
__device__ __forceinline__ uint32_t seen32(const AttendParams& p, int first, int keys, int pos, uint64_t w,
                                           int key0)
{
    // the keys below x, cut to these 32
    auto below = [&](int x) { return (uint32_t)((1ull << max(0, min(x - key0, 32))) - 1); };
    uint32_t see = below(p.tree ? keys : min(keys, pos + 1));
    if (p.window > 0)
        see &= ~below(pos - p.window + 1) | below(p.sinks);
    if (p.tree) {
        const int j = key0 - first;                     // new token of the first of the keys
        uint64_t t = j <= -32 ? ~0ull : j < 0 ? (w << -j) | ((1ull << -j) - 1) : j < 64 ? w >> j : 0;
        see &= (uint32_t)t;
    }
    return see;
}

// The new token of an item's row (a division by the group, in two instructions: code
// that runs once an item is not in the instruction cache, and costs by its length).
__device__ __forceinline__ int token_of(const AttendParams& p, int row)
{
    return (int)(__umulhi(2u * (uint32_t)row, p.group_mul) >> p.group_shift);
}

// 32 bytes to a 32-byte-aligned address: a whole sector by one thread.
__device__ __forceinline__ void store32(void* d, const uint32_t* r)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(d), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// `bytes` of global memory to shared memory.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint32_t load4(uint32_t at)
{
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(r) : "r"(at) : "memory");
    return r;
}

__device__ __forceinline__ uint2 load8(uint32_t at)
{
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
    return r;
}

__device__ __forceinline__ void load16(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

// 16 bytes to shared memory.
__device__ __forceinline__ void store16(uint32_t at, const uint32_t (&r)[4])
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// Stores N 16-bit values (packed in pairs) of an output row, as wide as its
// address allows.
template <int N>
__device__ __forceinline__ void store_row(uint16_t* d, const uint32_t* r)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(d);
    if (N % 16 == 0 && (a & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
            store32(d + 16 * k, r + 8 * k);
    } else if (N % 8 == 0 && (a & 15) == 0) {
#pragma unroll
        for (int k = 0; k < N / 8; ++k)
            reinterpret_cast<uint4*>(d)[k] = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
    } else if ((a & 3) == 0) {
#pragma unroll
        for (int k = 0; k < N / 2; ++k)
            reinterpret_cast<uint32_t*>(d)[k] = r[k];
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            d[k] = (uint16_t)(r[k >> 1] >> (16 * (k & 1)));
    }
}

// The natural log of a row's sum relative to 2^top.
__device__ __forceinline__ float lse_of(float top, float sum)
{
    return sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945f;
}

// Writes a row's four elements from 4 d4 on (o / sum, rounded once), and with
// the first of them its lse.  A row that saw nothing (sum 0) gets 0.  `sum` adds the
// probabilities as they entered the product with V, so that a row that one key
// dominates gets that key's value; `exact` adds them unrounded, for the lse.
template <int DT>
__device__ __forceinline__ void finish4(const AttendParams& p, const Request& q, int kv_head, int row,
                                        int d4, float4 o, float top, float sum, float exact)
{
    const int i = token_of(p, row), g = row - i * p.group;
    const int64_t tok = q.q0 + i;
    const int head = kv_head * p.group + g;
    const float f = 1.f / sum;
    const uint32_t r[2] = {sum == 0.f ? 0u : pack2<DT>(o.x * f, o.y * f),
                           sum == 0.f ? 0u : pack2<DT>(o.z * f, o.w * f)};
    store_row<4>(p.out + tok * p.out_token + (int64_t)head * p.out_head + d4 * 4, r);
    if (p.lse && d4 == 0)
        p.lse[tok * p.heads + head] = lse_of(top, exact);
}

// ---- work items ----
//
// An item is a tile of up to ROWS rows of a request (new token times query head
// of the group) and a key/value head, over the blocks of KEYS keys that some row
// of the tile sees, at least one (an empty row has an output too): those of the sinks,
// and those from the first window on.  Its cost in
// units: EXTRA for its queries and results, and NARROW for each block, or WIDE where
// the tile has more than SINGLE rows.  The units of the batch form one sequence
// -- request by request, tile by tile, head by head -- of which every CTA takes
// an equal contiguous share; a block belongs to the share that holds its first
// unit.  The host refuses batches of 2^32 units and more.
template <int ROWS_, int KEYS_, int EXTRA_, int NARROW = 1, int WIDE = NARROW, int SINGLE = ROWS_>
struct Shape {
    static constexpr int ROWS = ROWS_, KEYS = KEYS_, EXTRA = EXTRA_;
    static __device__ __forceinline__ int weight(int rows) { return rows > SINGLE ? WIDE : NARROW; }
    // k units in blocks, rounded up
    static __device__ __forceinline__ int blocks(int rows, int k)
    {
        return rows > SINGLE ? (k + WIDE - 1) / WIDE : (k + NARROW - 1) / NARROW;
    }
};

struct Tile {
    int row0, rows;        // its rows
    int lo, hi;            // keys they can see, beside the sinks
    int near, gap;         // blocks of the sinks; blocks left out behind them
    int blocks;
    unsigned units;
};

template <typename S>
__device__ __forceinline__ int tiles_of(const AttendParams& p, const Request& q)
{
    return (int)(((int64_t)q.n * p.group + S::ROWS - 1) / S::ROWS);
}

template <typename S>
__device__ __forceinline__ Tile tile_of(const AttendParams& p, const Request& q, int t)
{
    Tile x;
    x.row0 = t * S::ROWS;
    x.rows = min(S::ROWS, q.n * p.group - x.row0);
    key_range(p, q, token_of(p, x.row0), token_of(p, x.row0 + x.rows - 1), x.lo, x.hi);
    // (a window that reaches the sinks' last block leaves no block out)
    x.near = x.lo > 0 ? (min(p.sinks, x.hi) + S::KEYS - 1) / S::KEYS : 0;
    x.gap = max(0, x.lo / S::KEYS - x.near);
    x.blocks = max(1, x.near + max(0, (x.hi + S::KEYS - 1) / S::KEYS - x.near - x.gap));
    x.units = S::EXTRA + (unsigned)(S::weight(x.rows) * x.blocks);
    return x;
}

// Where a CTA's share begins: kept in shared memory for the CTA's roles.
struct Start {
    Request q;
    unsigned total, item;  // units of the batch; the first unit of the share's first item
    int ctas;              // CTAs that share them
    int r, tile, head;
};

// Run by one warp of CTA c: at most max_ctas CTAs with min_units each.  Few requests
// have several lanes each, which take their tiles in turn.
template <typename S>
__device__ __forceinline__ void find_start(const AttendParams& p, int lane, unsigned max_ctas,
                                           unsigned min_units, unsigned c, Start* out)
{
    int shift = 5;                                       // 2^shift requests at a time
    while (shift > 0 && p.batch.requests <= 1 << (shift - 1))
        --shift;
    const int at_once = 1 << shift, sub = lane >> shift, subs = 32 >> shift;
    auto units_of = [&](int r, Request& q) {             // of request r + lane % at_once
        r += lane & (at_once - 1);
        unsigned n = 0;
        if (r < p.batch.requests) {
            q = request_of(p, r);
            const int tiles = tiles_of<S>(p, q);
            for (int t = sub; t < tiles; t += subs)
                n += tile_of<S>(p, q, t).units;
        }
        for (int d = at_once; d < 32; d <<= 1)
            n += __shfl_xor_sync(0xffffffffu, n, d);
        return n * (unsigned)p.kv.heads;
    };
    Request q, q0;
    const unsigned v0 = units_of(0, q0);
    unsigned total = __reduce_add_sync(0xffffffffu, sub == 0 ? v0 : 0u);
    for (int r0 = at_once; r0 < p.batch.requests; r0 += at_once) {
        const unsigned v = units_of(r0, q);
        total += __reduce_add_sync(0xffffffffu, sub == 0 ? v : 0u);
    }
    const unsigned want = (total + min_units - 1) / min_units;
    const unsigned n = want < max_ctas ? want : max_ctas;
    if (lane == 0) {
        out->total = total;
        out->ctas = (int)n;
    }
    if (c >= n)
        return;
    const unsigned per = total / n, rem = total - per * n;
    const unsigned first = c * per + min(c, rem);
    unsigned base = 0;
    for (int r0 = 0; r0 < p.batch.requests; r0 += at_once) {
        unsigned v = v0;
        q = q0;
        if (r0 > 0)
            v = units_of(r0, q);
        unsigned sum = sub == 0 ? v : 0u;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const unsigned o = __shfl_up_sync(0xffffffffu, sum, d);
            sum += lane >= d ? o : 0;
        }
        unsigned at = base + sum - v;
        const unsigned here = __ballot_sync(0xffffffffu, sub == 0 && v && at <= first && first - at < v);
        base += __shfl_sync(0xffffffffu, sum, 31);
        if (!here)
            continue;
        // the request is found: its tiles, 32 at a time
        const int from = __ffs(here) - 1;
        Request f;
        f.q0 = __shfl_sync(0xffffffffu, q.q0, from);
        f.n = __shfl_sync(0xffffffffu, q.n, from);
        f.kv = __shfl_sync(0xffffffffu, q.kv, from);
        f.first = __shfl_sync(0xffffffffu, q.first, from);
        f.keys = __shfl_sync(0xffffffffu, q.keys, from);
        at = __shfl_sync(0xffffffffu, at, from);
        const int tiles = tiles_of<S>(p, f);
        for (int t0 = 0; t0 < tiles; t0 += 32) {
            const unsigned units = t0 + lane < tiles ? tile_of<S>(p, f, t0 + lane).units : 0;
            const unsigned w = units * (unsigned)p.kv.heads;
            unsigned upto = w;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned o = __shfl_up_sync(0xffffffffu, upto, d);
                upto += lane >= d ? o : 0;
            }
            const unsigned mine = at + upto - w;
            if (w && mine <= first && first - mine < w) {
                const unsigned head = (first - mine) / units;
                out->q = f;
                out->r = r0 + from;
                out->tile = t0 + lane;
                out->head = (int)head;
                out->item = mine + head * units;
            }
            at += __shfl_sync(0xffffffffu, upto, 31);
            if (at > first)
                break;
        }
        break;
    }
}

// A role's walk over the items of its CTA's share.
template <typename S>
struct Walk {
    const AttendParams& p;
    Request q;
    Tile x;
    unsigned u, u_end, per, rem, item;
    int r, t, tiles, head;
    int b_first, b_last;   // blocks of the item in this share

    __device__ Walk(const AttendParams& p_, const Start& s, unsigned c)
        : p(p_), q(s.q), item(s.item), r(s.r), t(s.tile), head(s.head)
    {
        per = s.total / (unsigned)s.ctas;
        rem = s.total - per * (unsigned)s.ctas;
        u = c * per + min(c, rem);
        u_end = u + per + (c < rem);
        tiles = tiles_of<S>(p, q);
        x = tile_of<S>(p, q, t);
        b_first = b_last = -1;
    }
    // the CTA whose share holds unit v
    __device__ int cta_of(unsigned v) const
    {
        const unsigned big = rem * (per + 1);
        return (int)(v < big ? v / (per + 1) : rem + (v - big) / per);
    }
    // blocks of the item whose first unit lies before unit v of it
    __device__ int blocks_before(unsigned v) const
    {
        const int k = (int)v - S::EXTRA;
        return k <= 0 ? 0 : min(S::blocks(x.rows, k), x.blocks);
    }
    // The next item with a block in the share.
    __device__ bool next()
    {
        do {
            if (u >= u_end)
                return false;
            if (u >= item + x.units) {
                item += x.units;
                if (++head == p.kv.heads) {
                    head = 0;
                    if (++t == tiles) {
                        t = 0;
                        do {
                            q = request_of(p, ++r);      // units remain, so a request does
                            tiles = tiles_of<S>(p, q);
                        } while (tiles == 0 && r + 1 < p.batch.requests);
                    }
                    x = tile_of<S>(p, q, t);
                }
            }
            b_first = blocks_before(u - item);
            b_last = blocks_before(min(x.units, u_end - item));
            u = item + min(x.units, u_end - item);
        } while (b_first == b_last);
        return true;
    }
    __device__ bool whole() const { return b_first == 0 && b_last == x.blocks; }
    __device__ int first_cta() const { return cta_of(item + S::EXTRA); }
    __device__ int last_cta() const
    {
        return cta_of(item + S::EXTRA + (unsigned)(S::weight(x.rows) * (x.blocks - 1)));
    }
    __device__ int key0(int b) const { return (b < x.near ? b : b + x.gap) * S::KEYS; }
};

// A partial result's item, for the kernel that joins them: written by the CTA
// the item starts in (rows 0: no item starts there and goes on).
struct alignas(32) JoinItem {
    int q0, row0, rows, kv_head, parts;
};

// Partial results of an item: slot 2 c + 1 of the CTA c0 it starts in, slot 2 c
// of the others; a slot holds o [ROWS][D], the reference maxima [ROWS] and the
// sums [ROWS] of rounded and of exact probabilities.  join_parts adds them in CTA order, by THREADS threads (tid) that
// meet at named barrier 1.  The parts come from L2, about 0.7 us away, so each
// of the three steps has all its loads in flight at once: the maxima and sums,
// the factors of every part (in `scratch`, `cap` >= 2 parts + 3 floats of shared
// memory), and 16 loads a thread of the results.
template <int DT, int D, int ROWS, int THREADS>
__device__ __forceinline__ void join_parts(const AttendParams& p, const Request& q, int kv_head,
                                           int row0, int rows, int c0, int c1, int tid,
                                           float* scratch, int cap)
{
    const int parts = c1 - c0 + 1;
    auto part = [&](int k) {
        return p.partial + (size_t)(2 * (c0 + k) + (k == 0)) * (ROWS * (D + 3));
    };
    const int step = min(rows, cap / (2 * parts + 3));   // rows at a time (at most kAttendMaxCtas parts)
    for (int r0 = 0; r0 < rows; r0 += step) {
        const int n = min(step, rows - r0);
        float* f = scratch;                              // [parts][n] maxima, then factors
        float* s = f + parts * n;                        // [parts][n] sums
        float* tops = s + parts * n;                     // [n], and the joined sums, twice [n]
        for (int i = tid; i < parts * n; i += THREADS) {
            const int k = i / n, r = i - k * n;
            f[i] = __ldcg(part(k) + ROWS * D + r0 + r);
            s[i] = __ldcg(part(k) + ROWS * (D + 1) + r0 + r);
        }
        named_bar_sync(1, THREADS);
        // a row's factors: by one thread, or by a warp if the parts are many
        const int lanes = parts > 8 ? 32 : 1, lane = tid & (lanes - 1);
        for (int r = tid / lanes; r < n; r += THREADS / lanes) {
            float top = -INFINITY, sum = 0.f, exact = 0.f;
            for (int k = lane; k < parts; k += lanes)
                top = fmaxf(top, f[k * n + r]);
            for (int d = lanes >> 1; d > 0; d >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            for (int k = lane; k < parts; k += lanes) {
                const float m = f[k * n + r], w = m == -INFINITY ? 0.f : ex2(m - top);
                f[k * n + r] = w;
                sum += w * s[k * n + r];
                if (p.lse)
                    exact += w * __ldcg(part(k) + ROWS * (D + 2) + r0 + r);
            }
            for (int d = lanes >> 1; d > 0; d >>= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, d);
                exact += __shfl_xor_sync(0xffffffffu, exact, d);
            }
            if (lane == 0) {
                tops[r] = top;
                tops[n + r] = sum;
                tops[2 * n + r] = exact;
            }
        }
        named_bar_sync(1, THREADS);
        constexpr int U = 8;
        const int tasks = n * (D / 4);
        for (int i = tid; i < tasks; i += U * THREADS) {
            float4 o[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < parts; k += 2) {
                const float* src[2] = {part(k) + (size_t)r0 * D, part(min(k + 1, parts - 1)) + (size_t)r0 * D};
                float4 a[2][U];
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (i + u * THREADS < tasks)
                            a[v][u] = __ldcg(reinterpret_cast<const float4*>(src[v]) + i + u * THREADS);
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (i + u * THREADS < tasks && k + v < parts) {
                            const float w = f[(k + v) * n + (i + u * THREADS) / (D / 4)];
                            o[u].x += w * a[v][u].x, o[u].y += w * a[v][u].y;
                            o[u].z += w * a[v][u].z, o[u].w += w * a[v][u].w;
                        }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * THREADS < tasks) {
                    const int r = (i + u * THREADS) / (D / 4);
                    finish4<DT>(p, q, kv_head, row0 + r0 + r, (i + u * THREADS) % (D / 4), o[u],
                                tops[r], tops[n + r], tops[2 * n + r]);
                }
        }
        named_bar_sync(1, THREADS);                      // scratch is free again
    }
}

}  // namespace att
}  // namespace lbv

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

// Bounded wait (about a second of SM cycles): false if it gave up.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity)
{
    if (mbar_try(bar, parity))
        return true;
    const long long t0 = clock64();
    while (!mbar_try(bar, parity))
        if (clock64() - t0 > (1ll << 31))
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

template <int DT>
__device__ __forceinline__ uint16_t pack1(float x)
{
    if constexpr (DT == LBV_F16)
        return __half_as_ushort(__float2half_rn(x));
    else
        return __bfloat16_as_ushort(__float2bfloat16_rn(x));
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

// Keys [lo, hi) that new tokens i0..i1 of a request can see.
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
    return s && key < q.keys && (p.window <= 0 || key > pos - p.window);
}

// The same for 32 keys from key0 on, as bits.
__device__ __forceinline__ uint32_t seen32(const AttendParams& p, const Request& q, int pos, uint64_t w,
                                           int key0)
{
    // keys [lo, hi) relative to key0, cut to 0..32
    int hi = (p.tree ? q.keys : min(q.keys, pos + 1)) - key0;
    int lo = p.window > 0 ? pos - p.window + 1 - key0 : 0;
    hi = max(0, min(hi, 32));
    lo = max(0, min(lo, 32));
    uint32_t see = (uint32_t)((1ull << hi) - 1) & ~(uint32_t)((1ull << lo) - 1);
    if (p.tree) {
        const int j = key0 - q.first;                   // new token of the first of the keys
        uint64_t t = j <= -32 ? ~0ull : j < 0 ? (w << -j) | ((1ull << -j) - 1) : j < 64 ? w >> j : 0;
        see &= (uint32_t)t;
    }
    return see;
}

// Stores N 16-bit values (packed in pairs) of an output row, as wide as its
// address allows.
template <int N>
__device__ __forceinline__ void store_row(uint16_t* d, const uint32_t* r)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(d);
    if (N % 8 == 0 && (a & 15) == 0) {
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
// the first of them its lse.  A row that saw nothing (sum 0) gets 0.
template <int DT>
__device__ __forceinline__ void finish4(const AttendParams& p, const Request& q, int kv_head, int row,
                                        int d4, float4 o, float top, float sum)
{
    const int i = row / p.group, g = row - i * p.group;
    const int64_t tok = q.q0 + i;
    const int head = kv_head * p.group + g;
    const float f = 1.f / sum;
    const uint32_t r[2] = {sum == 0.f ? 0u : pack2<DT>(o.x * f, o.y * f),
                           sum == 0.f ? 0u : pack2<DT>(o.z * f, o.w * f)};
    store_row<4>(p.out + tok * p.out_token + (int64_t)head * p.out_head + d4 * 4, r);
    if (p.lse && d4 == 0)
        p.lse[tok * p.heads + head] = lse_of(top, sum);
}

// Partial results of an item: slot 2 c + 1 of the CTA c0 it starts in, slot 2 c
// of the others; a slot holds o [ROWS][D], the reference maxima [ROWS] and the
// sums [ROWS].  join_parts adds them in CTA order, by the threads tid < threads.
template <int DT, int D, int ROWS>
__device__ __forceinline__ void join_parts(const AttendParams& p, const Request& q, int kv_head,
                                           int row0, int rows, int c0, int c1, int tid, int threads)
{
    auto part = [&](int c) {
        return p.partial + (size_t)(2 * c + (c == c0)) * (ROWS * (D + 2));
    };
    for (int i = tid; i < rows * (D / 4); i += threads) {
        const int row = i / (D / 4), d4 = i % (D / 4);
        float top = -INFINITY;
#pragma unroll 4
        for (int c = c0; c <= c1; ++c)
            top = fmaxf(top, __ldcg(part(c) + ROWS * D + row));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
            const float* s = part(c);
            const float m = __ldcg(s + ROWS * D + row);
            const float f = m == -INFINITY ? 0.f : ex2(m - top);
            const float4 a = __ldcg(reinterpret_cast<const float4*>(s + row * D + d4 * 4));
            sum += f * __ldcg(s + ROWS * (D + 1) + row);
            o.x += f * a.x, o.y += f * a.y, o.z += f * a.z, o.w += f * a.w;
        }
        finish4<DT>(p, q, kv_head, row0 + row, d4, o, top, sum);
    }
}

}  // namespace att
}  // namespace lbv

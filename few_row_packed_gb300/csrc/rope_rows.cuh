// rope_rows.cuh -- what the two appends share: the rows' elements, and where a new
// token's keys and values go.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "step_internal.h"

namespace lbv {
namespace rope {

template <int DT>
__device__ __forceinline__ float to_f32(uint16_t x)
{
    if constexpr (DT == LBV_F16)
        return __half2float(__ushort_as_half(x));
    else
        return __bfloat162float(__ushort_as_bfloat16(x));
}

template <int DT>
__device__ __forceinline__ uint16_t from_f32(float x)
{
    if constexpr (DT == LBV_F16)
        return __half_as_ushort(__float2half_rn(x));
    else
        return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <int SRC, bool VEC>
__device__ __forceinline__ void load4(const void* base, int64_t at, float (&x)[4])
{
    if constexpr (SRC == LBV_F32) {
        const float* s = static_cast<const float*>(base) + at;
        if constexpr (VEC) {
            const float4 v = *reinterpret_cast<const float4*>(s);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = s[i];
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(base) + at;
        if constexpr (VEC) {
            const ushort4 v = *reinterpret_cast<const ushort4*>(s);
            x[0] = to_f32<SRC>(v.x), x[1] = to_f32<SRC>(v.y);
            x[2] = to_f32<SRC>(v.z), x[3] = to_f32<SRC>(v.w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = to_f32<SRC>(s[i]);
        }
    }
}

template <int DST, bool VEC>
__device__ __forceinline__ void store4(uint16_t* d, const float (&x)[4])
{
    if constexpr (VEC) {
        *reinterpret_cast<ushort4*>(d) = make_ushort4(from_f32<DST>(x[0]), from_f32<DST>(x[1]),
                                                      from_f32<DST>(x[2]), from_f32<DST>(x[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] = from_f32<DST>(x[i]);
    }
}

// Where an item comes from and goes to.
struct Item {
    int which;             // 0 q, 1 k, 2 v
    int head;
    int o0, o1;            // offsets of its two groups of four elements
    int pair;              // first of its four pairs, -1: copied as it is
};

template <bool HALF>
__device__ __forceinline__ Item item_of(const RopeParams& p, int it, int per_head_shift)
{
    Item m;
    const int row = it >> per_head_shift;
    const int e = it - (row << per_head_shift);
    m.which = row < p.q_heads ? 0 : row < p.q_heads + p.kv.heads ? 1 : 2;
    m.head = m.which == 0 ? row : m.which == 1 ? row - p.q_heads : row - p.q_heads - p.kv.heads;
    m.pair = m.which < 2 && e < (p.rot >> 3) ? 4 * e : -1;
    m.o0 = HALF && m.pair >= 0 ? 4 * e : 8 * e;
    m.o1 = HALF && m.pair >= 0 ? (p.rot >> 1) + 4 * e : 8 * e + 4;
    return m;
}

// The request of token `tok` (-1: none) and its cache position, found by the whole
// block of THREADS threads into where[2] (shared memory).
template <int THREADS>
__device__ __forceinline__ void find_token(const lbv_batch& b, int tok, int* where)
{
    if (threadIdx.x == 0)
        where[0] = -1;
    __syncthreads();
    for (int r = threadIdx.x; r < b.requests; r += THREADS) {
        const int lo = b.q_start[r], hi = b.q_start[r + 1];
        if (lo <= tok && tok < hi) {
            where[0] = r;
            where[1] = b.kv_len[r] - hi + tok;
        }
    }
    __syncthreads();
}

// The page of position pos of request req, -1 if that slot does not exist.
__device__ __forceinline__ int page_of(const lbv_batch& b, const KvView& kv, int req, int pos)
{
    const int at = pos >> kv.page_shift;
    if (pos < 0 || at >= b.table_pages)
        return -1;
    const int page = b.block_table[(int64_t)req * b.table_stride + at];
    return page >= 0 && page < kv.pages ? page : -1;
}

// cos and sin of pair j at position `at`, times the factor.
__device__ __forceinline__ float2 turn_of(const RopeParams& p, int j, int at)
{
    const uint64_t f = (uint64_t)(int64_t)at * p.turns[j];
    float s, c;
    sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31 half turns
    return make_float2(c * p.factor, s * p.factor);
}

}  // namespace rope
}  // namespace lbv

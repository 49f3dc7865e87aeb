// rope_append.cu -- rotary positions of the new tokens' queries and keys, and
// the append of keys and values to the paged cache, in one pass.
//
// With t = position * f_j radians, pair (a, b) of a head becomes
//     a' = c (a cos t - b sin t),   b' = c (b cos t + a sin t)
// for the rotation's factor c.  Frequencies are kept as whole numbers F_j of
// 2^-64 turns, so position * F_j modulo 2^64 is the angle's fraction of a turn
// with no reduction error at any position; its top 32 bits go to sincospif,
// whose argument is then exact to 2^-24 of the angle.  (In fp32 the product
// position * f_j would be off by 0.004 radians at position 10^5.)
//
// Bound by memory: every element is read once (fp32 or 16 bit) and written
// once (16 bit), 4 flops a rotated element.  One block takes a token (or,
// with few tokens, a part of one): its threads put their first rows in flight,
// compute the token's cos and sin once for all heads, and then rotate.  A
// thread's item is two groups of four elements -- the two halves of four
// pairs, or eight neighbours -- so that loads are 16 (or 8) and stores 8 bytes
// wide.  8191 tokens of 48 + 8 + 8 heads of 128, fp32 to bf16: 61 us, 6.6 TB/s, 97 % of
// what a copy reaches; 8 tokens 2.4 us, 64 requests of 1 to 8 tokens 4.3 us, a launch and
// one round trip to memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "step_internal.h"

namespace lbv {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;             // items a thread keeps in flight

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

template <int SRC, int DST, bool HALF, bool VEC>
__global__ void __launch_bounds__(kThreads) lbv_rope_append_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ float2 turn[kMaxRot / 2];
    __shared__ int where[2];                       // request (-1: none), cache position
    const int tok = blockIdx.x;
    const int per_head_shift = p.kv.dim == 128 ? 4 : 3;
    const int total = (p.q_heads + 2 * p.kv.heads) << per_head_shift;
    const int step = kThreads * gridDim.y;
    const int first = blockIdx.y * kThreads + threadIdx.x;

    after_previous();
    float x0[kAhead][4], x1[kAhead][4];
    auto fetch = [&](int it, float (&a)[4], float (&b)[4]) {
        const Item m = item_of<HALF>(p, it, per_head_shift);
        const int64_t at = tok * p.src_token[m.which] + m.head * p.src_head[m.which];
        load4<SRC, VEC>(p.src[m.which], at + m.o0, a);
        load4<SRC, VEC>(p.src[m.which], at + m.o1, b);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (first + u * step < total)
            fetch(first + u * step, x0[u], x1[u]);

    if (threadIdx.x == 0)
        where[0] = -1;
    __syncthreads();
    for (int r = threadIdx.x; r < p.batch.requests; r += kThreads) {
        const int lo = p.batch.q_start[r], hi = p.batch.q_start[r + 1];
        if (lo <= tok && tok < hi) {
            where[0] = r;
            where[1] = p.batch.kv_len[r] - hi + tok;
        }
    }
    __syncthreads();
    const int req = where[0], pos = where[1];
    if (req < 0)
        return;                                    // a row of no request
    if (threadIdx.x < (p.rot >> 1)) {
        const int at = p.positions ? p.positions[tok] : pos;
        const uint64_t f = (uint64_t)(int64_t)at * p.turns[threadIdx.x];
        float s, c;
        sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31 half turns
        turn[threadIdx.x] = make_float2(c * p.factor, s * p.factor);
    }
    int64_t slot = -1;
    const int page_at = pos >> p.kv.page_shift;
    if (pos >= 0 && page_at < p.batch.table_pages) {
        const int page = p.batch.block_table[(int64_t)req * p.batch.table_stride + page_at];
        if (page >= 0 && page < p.kv.pages)
            slot = page * p.kv.page_stride +
                   (pos & ((1 << p.kv.page_shift) - 1)) * p.kv.token_stride;
    }
    __syncthreads();

    auto finish = [&](int it, float (&a)[4], float (&b)[4]) {
        const Item m = item_of<HALF>(p, it, per_head_shift);
        if (m.pair >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = turn[m.pair + i];
                float& x = HALF ? a[i] : i < 2 ? a[2 * i] : b[2 * i - 4];
                float& y = HALF ? b[i] : i < 2 ? a[2 * i + 1] : b[2 * i - 3];
                const float xn = x * t.x - y * t.y;
                y = y * t.x + x * t.y;
                x = xn;
            }
        }
        if (m.which == 0) {
            uint16_t* d = p.q_out + tok * p.out_token + m.head * p.out_head;
            store4<DST, VEC>(d + m.o0, a);
            store4<DST, VEC>(d + m.o1, b);
        } else if (slot >= 0) {
            uint16_t* d = (m.which == 1 ? p.kv.k : p.kv.v) + slot + m.head * p.kv.head_stride;
            store4<DST, true>(d + m.o0, a);
            store4<DST, true>(d + m.o1, b);
        }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (first + u * step < total)
            finish(first + u * step, x0[u], x1[u]);
    for (int it = first + kAhead * step; it < total; it += step) {
        fetch(it, x0[0], x1[0]);
        finish(it, x0[0], x1[0]);
    }
}

template <int SRC, int DST, bool HALF>
cudaError_t launch(const RopeParams& p, bool vec, cudaStream_t st)
{
    const int total = (p.q_heads + 2 * p.kv.heads) * (p.kv.dim / 8);
    // few tokens: one item a thread, so that the whole call is in flight at
    // once; many: kAhead items a thread
    const int per = p.batch.tokens < 256 ? 1 : kAhead;
    const dim3 grid((unsigned)p.batch.tokens,
                    (unsigned)((total + kThreads * per - 1) / (kThreads * per)));
    return vec ? launch_after(lbv_rope_append_kernel<SRC, DST, HALF, true>, grid, kThreads, 0, st, p)
               : launch_after(lbv_rope_append_kernel<SRC, DST, HALF, false>, grid, kThreads, 0, st, p);
}

template <int SRC>
cudaError_t launch_src(const RopeParams& p, lbv_dtype dst, lbv_rope_layout layout, bool vec,
                       cudaStream_t st)
{
    if (dst == LBV_F16)
        return layout == LBV_ROPE_HALF ? launch<SRC, LBV_F16, true>(p, vec, st)
                                       : launch<SRC, LBV_F16, false>(p, vec, st);
    return layout == LBV_ROPE_HALF ? launch<SRC, LBV_BF16, true>(p, vec, st)
                                   : launch<SRC, LBV_BF16, false>(p, vec, st);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, lbv_dtype src, lbv_dtype dst,
                               lbv_rope_layout layout, bool vec, cudaStream_t st)
{
    if (src == LBV_F32)
        return launch_src<LBV_F32>(p, dst, layout, vec, st);
    return src == LBV_F16 ? launch_src<LBV_F16>(p, dst, layout, vec, st)
                          : launch_src<LBV_BF16>(p, dst, layout, vec, st);
}

}  // namespace lbv

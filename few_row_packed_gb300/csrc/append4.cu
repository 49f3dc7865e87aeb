// append4.cu -- rotary positions of the new tokens, and the append to a cache of 4 bits.
//
// The rotation is that of rope_append.cu; a group x of 64 rotated elements is then held
// as codes of 4 bits between its bounds:
//     bias = round16(min x), scale = round16((max x - min x) * (1 / 15)),
//     code = round((x - bias) * (1 / scale)) in 0..15.
// Queries are items of two groups of four elements, as in rope_append.cu.  Of keys and values
// a thread has 8 neighbours, so a group of 64 is 8 lanes, whose minimum and maximum meet in three
// exchanges, and whose codes are 32 neighbouring bytes.  With halves that pair up it loads
// its elements' partners when it rotates them: they are another thread's own, so they
// come from L1, and any rotated part of a head is treated alike.
//
// A code is a decision: values that differ in their last bit may fall on two sides of a
// border.  So the arithmetic is that of elementary fp32 operations, the angle in
// radians and every product and sum rounded by itself: a program that follows the
// definition gets the same codes.  (The angle's fraction of a turn is exact to 2^-40 before
// that; its rounding to fp32 is off by up to 4e-7, a millionth of a step between codes.)
// Queries have no codes but the same turns, one table a token: 4e-7 of a query is 2^-21, where
// its rounding to 16 bits takes 2^-11 or 2^-8.
//
// Bound by memory: every element is read once, queries leave as 16 bits, keys and values as 4.5.
// 8191 tokens of 48 + 8 + 8 heads of 128, fp32 to bf16: 64 us, 5.9 TB/s, 87 % of what a copy
// reaches.  From bf16 56 us, 4.3 TB/s: there the instructions count, a third of them cos and sin by
// radians and the codes.  (With a thread for both halves of a head's pairs, eight neighbours
// each: 126 us from fp32.  With 256 threads a block, addresses and turns anew for every item and
// elements turned to fp32 as they are loaded, which waits for each item's loads: 70 and 92.)
#include <type_traits>

#include "kv4.cuh"
#include "rope_rows.cuh"

namespace lbv {

using namespace rope;

namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;             // items a thread keeps in flight (2: 17 %, 8: 4 % longer)
constexpr int kBlocks = 8;            // blocks an SM has room for in registers (left to the compiler: 4 % longer)

// cos and sin of pair j at position `at`, times the factor.
__device__ __forceinline__ float2 turn32_of(const RopeParams& p, int j, int at)
{
    const uint64_t f = (uint64_t)(int64_t)at * p.turns[j];
    const float angle = __fmul_rn(__ull2float_rn(f >> 24), (float)(6.283185307179586476925 / 1099511627776.0));
    return make_float2(__fmul_rn(cosf(angle), p.factor), __fmul_rn(sinf(angle), p.factor));
}

// a b - c d and a b + c d, each step rounded.
__device__ __forceinline__ float cross(float a, float b, float c, float d)
{
    return __fsub_rn(__fmul_rn(a, b), __fmul_rn(c, d));
}

__device__ __forceinline__ float dot(float a, float b, float c, float d)
{
    return __fadd_rn(__fmul_rn(a, b), __fmul_rn(c, d));
}

// Four elements as they are in memory: turned to fp32 where they are used, so that the loads of
// all items are under way before one is waited for.
template <int SRC>
using Raw = std::conditional_t<SRC == LBV_F32, float4, uint2>;

template <int SRC, bool VEC>
__device__ __forceinline__ Raw<SRC> load_raw(const void* base, int64_t at)
{
    if constexpr (SRC == LBV_F32) {
        const float* s = static_cast<const float*>(base) + at;
        return VEC ? *reinterpret_cast<const float4*>(s) : make_float4(s[0], s[1], s[2], s[3]);
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(base) + at;
        return VEC ? *reinterpret_cast<const uint2*>(s)
                   : make_uint2(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16);
    }
}

template <int SRC>
__device__ __forceinline__ void unpack(const Raw<SRC>& r, float* x)
{
    if constexpr (SRC == LBV_F32) {
        x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
    } else {
        x[0] = to_f32<SRC>((uint16_t)r.x), x[1] = to_f32<SRC>((uint16_t)(r.x >> 16));
        x[2] = to_f32<SRC>((uint16_t)r.y), x[3] = to_f32<SRC>((uint16_t)(r.y >> 16));
    }
}

template <int SRC, int DST, bool HALF, bool VEC>
__global__ void __launch_bounds__(kThreads, kBlocks) lbv_rope_append4_kernel(const __grid_constant__ RopeParams p)
{
    __shared__ float2 turn[kMaxRot / 2];
    __shared__ int where[2];                       // request (-1: none), cache position
    const int tok = blockIdx.x, lane = threadIdx.x & 31;
    const int per_head_shift = p.kv.dim == 128 ? 4 : 3;
    // items of queries, then, from a warp's first lane on, keys and values
    const int queries = p.q_heads << per_head_shift, keys = (queries + 31) & ~31;
    const int total = keys + (2 * p.kv.heads << per_head_shift);
    const int step = kThreads * gridDim.y;
    const int first = blockIdx.y * kThreads + threadIdx.x;
    // A thread's items are in one place of their heads: of a query, two groups of four; of a key
    // or value, eight neighbours.
    const int in_head = first & ((1 << per_head_shift) - 1), at = in_head * 8;
    const Item m = item_of<HALF>(p, in_head, per_head_shift);

    after_previous();
    Raw<SRC> x0[kAhead], x1[kAhead];
    // the head of an item of keys or values, which come after the keys
    auto row_of = [&](int it, int& which) {
        const int row = (it - keys) >> per_head_shift;
        which = row >= p.kv.heads ? 2 : 1;
        return row - (which - 1) * p.kv.heads;
    };
    auto fetch = [&](int it, Raw<SRC>& a, Raw<SRC>& b) {
        const bool query = it < keys;
        int which = 0;
        const int head = query ? it >> per_head_shift : row_of(it, which);
        const int64_t from = tok * p.src_token[which] + head * p.src_head[which];
        a = load_raw<SRC, VEC>(p.src[which], from + (query ? m.o0 : at));
        b = load_raw<SRC, VEC>(p.src[which], from + (query ? m.o1 : at + 4));
    };
    auto is = [&](int it) { return it < queries || (it >= keys && it < total); };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (is(first + u * step))
            fetch(first + u * step, x0[u], x1[u]);

    find_token<kThreads>(p.batch, tok, where);
    const int req = where[0], pos = where[1];
    if (req < 0)
        return;                                    // a row of no request
    if (threadIdx.x < (p.rot >> 1))
        turn[threadIdx.x] = turn32_of(p, threadIdx.x, p.positions ? p.positions[tok] : pos);
    const int page = page_of(p.batch, p.kv, req, pos);
    const int slot = pos & ((1 << p.kv.page_shift) - 1);
    __syncthreads();

    float2 turns[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        turns[i] = turn[max(m.pair, 0) + i];
    auto query = [&](int it, const Raw<SRC>& x0, const Raw<SRC>& x1) {
        float a[4], b[4];
        unpack<SRC>(x0, a);
        unpack<SRC>(x1, b);
        if (m.pair >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = turns[i];
                float& x = HALF ? a[i] : i < 2 ? a[2 * i] : b[2 * i - 4];
                float& y = HALF ? b[i] : i < 2 ? a[2 * i + 1] : b[2 * i - 3];
                const float xn = cross(x, t.x, y, t.y);
                y = dot(y, t.x, x, t.y);
                x = xn;
            }
        }
        uint16_t* d = p.q_out + tok * p.out_token + (it >> per_head_shift) * p.out_head;
        store4<DST, VEC>(d + m.o0, a);
        store4<DST, VEC>(d + m.o1, b);
    };
    // all lanes of a warp come here together; those past the last do nothing
    auto held = [&](int it, const Raw<SRC>& x0, const Raw<SRC>& x1) {
        const bool in = it < total;
        int which;
        const int head = row_of(in ? it : keys, which);
        float a[8];
        unpack<SRC>(x0, a);
        unpack<SRC>(x1, a + 4);
        if (in && which == 1 && at < p.rot) {
            const int half = p.rot >> 1;           // a multiple of 4
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int o = at + 4 * h;
                if constexpr (HALF) {
                    const bool low = o < half;
                    float b[4];
                    unpack<SRC>(load_raw<SRC, VEC>(p.src[1], tok * p.src_token[1] + head * p.src_head[1] +
                                                                 (low ? o + half : o - half)), b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = turn[(low ? o : o - half) + i];
                        float& v = a[4 * h + i];
                        v = low ? cross(v, t.x, b[i], t.y) : dot(v, t.x, b[i], t.y);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 t = turn[(o >> 1) + i];
                        float &v = a[4 * h + 2 * i], &w = a[4 * h + 2 * i + 1];
                        const float n = cross(v, t.x, w, t.y);
                        w = dot(w, t.x, v, t.y);
                        v = n;
                    }
                }
            }
        }
        // the group's bounds, by its 8 lanes
        constexpr float kMost = DST == LBV_F16 ? 32768.f : 8.5070591730234616e37f;    // 2^15, 2^126
        float lo = a[0], hi = a[0];
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, a[i]), hi = fmaxf(hi, a[i]);
            odd = odd || !(fabsf(a[i]) <= kMost);
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        }
        odd = (__ballot_sync(0xffffffffu, odd) >> (lane & 24)) & 0xFFu;
        if (!in || page < 0)
            return;
        uint16_t bias = from_f32<DST>(lo), scale = from_f32<DST>(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f));
        float s = to_f32<DST>(scale);
        if (!(s >= 1.17549435e-38f))               // its reciprocal would not be finite
            s = 0.f, scale = 0;
        const float low = to_f32<DST>(bias), inverse = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            word |= (uint32_t)max(0, min(15, __float2int_rn(__fmul_rn(__fsub_rn(a[i], low), inverse))))
                    << (4 * (i >> 1) + 16 * (i & 1));
        if (odd)
            scale = 0x7FFF;                        // NaN in both types
        const int cs = kv4::chunk_shift(p.kv), to = slot & ((1 << cs) - 1);
        const int planes = p.kv.dim >> 5, plane = (which - 1) * (planes >> 1) + (at >> 6);
        uint8_t* c = kv4::chunk(p.kv, page, head, slot);
        *reinterpret_cast<uint32_t*>(c + kv4::codes_at(plane, to, cs) + ((at >> 3) & 7) * 4) = word;
        if ((at & 63) == 0)
            *reinterpret_cast<uint32_t*>(c + kv4::scale_at(planes, plane, to, cs)) = scale | ((uint32_t)bias << 16);
    };
    auto finish = [&](int it, const Raw<SRC>& a, const Raw<SRC>& b) {
        if (it - lane >= keys)                     // a warp has either
            held(it, a, b);
        else if (it < queries)
            query(it, a, b);
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (first - lane + u * step < total)
            finish(first + u * step, x0[u], x1[u]);
    for (int it = first + kAhead * step; it - lane < total; it += step) {
        if (is(it))
            fetch(it, x0[0], x1[0]);
        finish(it, x0[0], x1[0]);
    }
}

template <int SRC, int DST, bool HALF>
cudaError_t launch(const RopeParams& p, bool vec, cudaStream_t st)
{
    const int total = (p.q_heads * (p.kv.dim / 8) + 31) / 32 * 32 + 2 * p.kv.heads * (p.kv.dim / 8);
    // few tokens: one item a thread, so that the whole call is in flight at once
    const int per = p.batch.tokens < 256 ? 1 : kAhead;
    const dim3 grid((unsigned)p.batch.tokens,
                    (unsigned)((total + kThreads * per - 1) / (kThreads * per)));
    return vec ? launch_after(lbv_rope_append4_kernel<SRC, DST, HALF, true>, grid, kThreads, 0, st, p)
               : launch_after(lbv_rope_append4_kernel<SRC, DST, HALF, false>, grid, kThreads, 0, st, p);
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

cudaError_t launch_rope_append4(const RopeParams& p, lbv_dtype src, lbv_dtype dst,
                                lbv_rope_layout layout, bool vec, cudaStream_t st)
{
    if (src == LBV_F32)
        return launch_src<LBV_F32>(p, dst, layout, vec, st);
    return src == LBV_F16 ? launch_src<LBV_F16>(p, dst, layout, vec, st)
                          : launch_src<LBV_BF16>(p, dst, layout, vec, st);
}

}  // namespace lbv

// attend_join.cu -- adds the partial results of items that several CTAs share.
// A CTA that joined its item by itself would read every part alone, at the
// latency of L2: 24 us for 20 parts of 48 rows, as long as the call's keys and
// values take, and 20 us for 2 parts of 256 rows.  This launch, which starts
// while the attention kernel drains, spreads the rows over the SMs.
//
// One warp a row, or four rows of two parts: its lanes take the parts' maxima and sums,
// then four elements each of the results.  The parts are added in CTA order.  Bound by
// round trips to L2 and the launch: 96 rows of some 19 parts take 5 us after the attention
// kernel's end (2 the launch, 2 to find the item, 1.5 the parts), 152 items of 256
// rows 9 (40 MB read).
#include <algorithm>

#include "attend_common.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kWarps = 4;

constexpr int kLook = 5;                         // items a lane looks at at a time
constexpr int kFew = 2, kAtOnce = 4;             // of kFew parts a warp takes kAtOnce rows at once

// DIRECT: the grid has a column for every CTA, else one for every divided item (few, of
// many parts).
template <int DT, int D, bool DIRECT>
__global__ void __launch_bounds__(kWarps * 32, DIRECT ? 6 : 2)
    lbv_attend_join_kernel(const __grid_constant__ AttendParams p, int slot_rows, int ctas)
{
    after_previous();
    // The next launch may take its places now.  (The attention kernels do not let this one
    // in before their end: its blocks would hold places beside them, 1.3 us more.)
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const JoinItem* items = static_cast<const JoinItem*>(p.items);
    auto load = [&](int c, int4& i, int& parts) {
        i = __ldcg(reinterpret_cast<const int4*>(items + c));
        parts = __ldcg(&items[c].parts);
    };
    JoinItem it;
    int c0 = -1;                                 // the CTA the item starts in
    int4 i;
    if (DIRECT) {
        c0 = blockIdx.x;
        load(c0, i, it.parts);
        if (i.z <= 0)
            return;
    } else {
        int before = 0;
        for (int b = 0; b < ctas && c0 < 0; b += 32 * kLook) {
            int4 look[kLook];
            int parts[kLook];
#pragma unroll
            for (int k = 0; k < kLook; ++k) {
                look[k] = make_int4(0, 0, 0, 0);
                parts[k] = 0;
                if (b + k * 32 + lane < ctas)
                    load(b + k * 32 + lane, look[k], parts[k]);
            }
#pragma unroll
            for (int k = 0; k < kLook; ++k) {
                const unsigned set = __ballot_sync(0xffffffffu, look[k].z > 0);
                const unsigned here = __ballot_sync(
                    0xffffffffu, look[k].z > 0 && before + __popc(set & ((1u << lane) - 1)) == (int)blockIdx.x);
                before += __popc(set);
                if (here) {
                    const int from = __ffs(here) - 1;
                    c0 = b + k * 32 + from;
                    i = make_int4(__shfl_sync(0xffffffffu, look[k].x, from), __shfl_sync(0xffffffffu, look[k].y, from),
                                  __shfl_sync(0xffffffffu, look[k].z, from), __shfl_sync(0xffffffffu, look[k].w, from));
                    it.parts = __shfl_sync(0xffffffffu, parts[k], from);
                }
            }
        }
        if (c0 < 0)
            return;
    }
    it.q0 = i.x, it.row0 = i.y, it.rows = i.z, it.kv_head = i.w;
    constexpr int LANES = D / 4;                 // lanes that hold a row
    constexpr int AT_ONCE = 32 / LANES;          // parts a load takes
    const int sub = lane / LANES, d4 = lane % LANES;
    Request q;
    q.q0 = it.q0;
    const size_t slot = (size_t)slot_rows * (D + 3);
    auto part = [&](int k) {
        return p.partial + (size_t)(2 * (c0 + k) + (k == 0)) * slot;
    };
    if (it.parts <= kFew) {
        // their results, and by lane kFew r + k the maximum and the sums of row r in part k
        for (int row0 = (blockIdx.y * kWarps + warp) * kAtOnce; row0 < it.rows;
             row0 += gridDim.y * kWarps * kAtOnce) {
            constexpr int LOADS = kFew / AT_ONCE;
            float4 a[kAtOnce][LOADS];
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r)
#pragma unroll
                for (int j = 0; j < LOADS; ++j)
                    if (row0 + r < it.rows && j * AT_ONCE + sub < it.parts)
                        a[r][j] = __ldcg(reinterpret_cast<const float4*>(part(j * AT_ONCE + sub) + (row0 + r) * D) + d4);
            const int my = row0 + lane / kFew, k = lane % kFew;
            float m = -INFINITY, s = 0.f, x = 0.f;
            if (lane < kFew * kAtOnce && my < it.rows && k < it.parts) {
                m = __ldcg(part(k) + slot_rows * D + my);
                s = __ldcg(part(k) + slot_rows * (D + 1) + my);
                x = __ldcg(part(k) + slot_rows * (D + 2) + my);
            }
            const float top = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const float w = m == -INFINITY ? 0.f : ex2(m - top);
            float sum = w * s, exact = w * x;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            exact += __shfl_xor_sync(0xffffffffu, exact, 1);
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int j = 0; j < LOADS; ++j) {
                    const float f = __shfl_sync(0xffffffffu, w, r * kFew + j * AT_ONCE + sub);
                    if (row0 + r < it.rows && j * AT_ONCE + sub < it.parts)
                        o.x += f * a[r][j].x, o.y += f * a[r][j].y, o.z += f * a[r][j].z, o.w += f * a[r][j].w;
                }
                if constexpr (AT_ONCE == 2) {
                    o.x += __shfl_xor_sync(0xffffffffu, o.x, 16), o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
                    o.z += __shfl_xor_sync(0xffffffffu, o.z, 16), o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
                }
                const float t = __shfl_sync(0xffffffffu, top, r * kFew), l = __shfl_sync(0xffffffffu, sum, r * kFew),
                            e = __shfl_sync(0xffffffffu, exact, r * kFew);
                if (sub == 0 && row0 + r < it.rows)
                    finish4<DT>(p, q, it.kv_head, it.row0 + row0 + r, d4, o, t, l, e);
            }
        }
        return;
    }
    for (int row = blockIdx.y * kWarps + warp; row < it.rows; row += gridDim.y * kWarps) {
        // the first parts' results, maxima and sums in one round of loads
        constexpr int AHEAD = DIRECT ? 8 : 20 / AT_ONCE;
        float4 first[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j)
            if (j * AT_ONCE + sub < it.parts)
                first[j] = __ldcg(reinterpret_cast<const float4*>(part(j * AT_ONCE + sub) + row * D) + d4);
        float m = -INFINITY, s = 0.f, x = 0.f;   // of the lane's part
        if (lane < it.parts) {
            m = __ldcg(part(lane) + slot_rows * D + row);
            s = __ldcg(part(lane) + slot_rows * (D + 1) + row);
            x = __ldcg(part(lane) + slot_rows * (D + 2) + row);
        }
        float top = m;
        for (int k = lane + 32; k < it.parts; k += 32)
            top = fmaxf(top, __ldcg(part(k) + slot_rows * D + row));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        float w = m == -INFINITY ? 0.f : ex2(m - top), sum = w * s, exact = w * x;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float f, float4 a) {
            o.x += f * a.x, o.y += f * a.y, o.z += f * a.z, o.w += f * a.w;
        };
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const float f = __shfl_sync(0xffffffffu, w, (j * AT_ONCE + sub) & 31);
            if (j * AT_ONCE + sub < it.parts)
                add(f, first[j]);
        }
        for (int k0 = 0; k0 < it.parts; k0 += 32) {
            if (k0 > 0) {
                const int k = k0 + lane;
                w = 0.f;
                if (k < it.parts) {
                    const float n = __ldcg(part(k) + slot_rows * D + row);
                    w = n == -INFINITY ? 0.f : ex2(n - top);
                    sum += w * __ldcg(part(k) + slot_rows * (D + 1) + row);
                    exact += w * __ldcg(part(k) + slot_rows * (D + 2) + row);
                }
            }
            const int n = min(32, it.parts - k0);
#pragma unroll 8
            for (int j = k0 > 0 ? 0 : AHEAD * AT_ONCE; j < n; j += AT_ONCE) {
                const float f = __shfl_sync(0xffffffffu, w, j + sub);
                if (j + sub < n)
                    add(f, __ldcg(reinterpret_cast<const float4*>(part(k0 + j + sub) + row * D) + d4));
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            exact += __shfl_xor_sync(0xffffffffu, exact, d);
        }
        if constexpr (AT_ONCE == 2) {
            o.x += __shfl_xor_sync(0xffffffffu, o.x, 16), o.y += __shfl_xor_sync(0xffffffffu, o.y, 16);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, 16), o.w += __shfl_xor_sync(0xffffffffu, o.w, 16);
        }
        if (sub == 0)
            finish4<DT>(p, q, it.kv_head, it.row0 + row, d4, o, top, sum, exact);
    }
}

template <int DT, int D>
cudaError_t launch(const AttendParams& p, int slot_rows, int ctas, cudaStream_t st)
{
    // divided items: no more than there are items, or CTAs
    const int64_t items = ((int64_t)p.batch.tokens * p.group / slot_rows + p.batch.requests) * p.kv.heads;
    // A column for every CTA where the items have up to eight parts on average, else for
    // every item; blocks for the rows of an item of twice the average (more are taken in
    // turn).  Blocks without work cost too: with a column for each of 106 undivided items and
    // 32 blocks for the largest slot, the launch took 28 us.
    const bool direct = items * 8 >= ctas;
    const int64_t rows = std::min<int64_t>(slot_rows, 2 * attend_average_rows(p));
    const int per = slot_rows <= 64 ? kWarps : kWarps * (direct ? kAtOnce : 2);
    const dim3 grid((unsigned)(direct ? ctas : items), (unsigned)((rows + per - 1) / per));
    return launch_after(direct ? lbv_attend_join_kernel<DT, D, true> : lbv_attend_join_kernel<DT, D, false>, grid,
                        kWarps * 32, 0, st, p, slot_rows, ctas);
}

}  // namespace

cudaError_t launch_attend_join(const AttendParams& p, lbv_dtype dt, int slot_rows, int ctas,
                               cudaStream_t st)
{
    if (dt == LBV_F16)
        return p.kv.dim == 128 ? launch<LBV_F16, 128>(p, slot_rows, ctas, st)
                               : launch<LBV_F16, 64>(p, slot_rows, ctas, st);
    return p.kv.dim == 128 ? launch<LBV_BF16, 128>(p, slot_rows, ctas, st)
                           : launch<LBV_BF16, 64>(p, slot_rows, ctas, st);
}

// Whether the few-row kernel leaves its parts to this launch: where the items
// (row tiles times kv heads, estimated from the batch's counts) have four CTAs
// each or more.  Elsewhere the last CTA of an item joins its two or three parts
// of 16 rows in less time than a launch takes.
bool attend_joins_apart(const AttendParams& p, int tile_rows, int ctas)
{
    const int64_t rows = (int64_t)p.batch.tokens * p.group;
    const int64_t tiles = (rows + tile_rows - 1) / tile_rows;
    const int64_t items = (tiles > p.batch.requests ? tiles : p.batch.requests) * p.kv.heads;
    return ctas >= 4 * items;
}

}  // namespace lbv

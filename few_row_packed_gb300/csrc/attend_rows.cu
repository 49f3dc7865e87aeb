// attend_rows.cu -- attention of few new tokens over the paged cache (plain
// decoding, verify calls, trees of drafted tokens): memory-bound.
//
//     o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(t_ij - m_i),
//     t_ij = scale log2(e) q_i . k_j
// over the keys j that row i sees, with a running reference m_i.  Changing m_i
// rescales what was summed, so it only moves when a block's maximum passes it
// by more than 8 (p stays below 2^8, in fp32 sums and 16-bit operands alike).
//
// The rows of one work item are the new tokens of a request times the query
// heads that share a key/value head, so every key and value is read from
// memory once for all of them.  Bound by that read: 4 D bytes a key and
// key/value head.
//   * Keys come in blocks of 64.  All (item, block) pairs of the batch form one
//     sequence, of which each CTA of a resident grid takes an equal contiguous
//     share: ragged contexts and few long ones load the SMs alike.  An item
//     whose blocks lie in several CTAs leaves partial results (m, sum, o) in the
//     workspace; the CTA that arrives last adds them in CTA order, so the
//     result does not depend on timing.
//   * A producer warp (its warpgroup gives its registers to the others) copies blocks with TMA (a box is 64 elements of a head
//     times the slots of a page in the block) into a ring of 128-byte-swizzled
//     stages, so that ldmatrix reads them without bank conflicts.
//   * Four warps take 16 keys each of a block (WM > 1: as many sets of them
//     share the rows): mma.sync m16n8k16 with the rows as M.  A tile of 16 rows
//     is the natural size of a verify call; the 128-row tiles of tcgen05 would
//     be mostly padding.  The warps' results meet in shared memory once per
//     item.
#include "attend_common.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kBlock = 64;                       // keys per block
constexpr int kKeyWarps = 4;
// Units of an item beside its blocks, and the least share of a CTA (below, joining
// costs more than it saves).
constexpr int kExtra = 1, kMinUnits = 2;

template <int D, int MT, int WM>
struct Geo {
    static constexpr int ROWS = 16 * MT * WM;
    static constexpr int WARPS = kKeyWarps * WM;
    static constexpr int THREADS = WARPS * 32 + 128;        // the producer's warpgroup first
    static constexpr int HALF = kBlock * 128;               // 64 elements of 64 keys
    static constexpr int STAGE = 2 * (D / 64) * HALF;       // K then V
    // about 96 KB of ring where two CTAs share an SM, else 160
    static constexpr int CTAS = WM == 1 ? 2 : 1;
    // Registers a thread after the warpgroups' split.  The launch holds 128
    // (256 threads, two CTAs) or 168 (384 threads) times its threads:
    // 128 * 256 = 40 * 128 + 216 * 128, 168 * 384 = 40 * 128 + 232 * 256.
    static constexpr int REGS_PRODUCER = 40, REGS_ROWS = WM == 1 ? 216 : 232;
    static constexpr int NST = (CTAS == 2 ? 98304 : 163840) / STAGE;
    static constexpr int OLD = D + 4;                       // floats per row of the join buffer
    static constexpr int SLOT = ROWS * (D + 2);             // floats of one partial result
    // shared memory
    static constexpr int O_BUF = NST * STAGE;
    static constexpr int M_BUF = O_BUF + ROWS * OLD * 4;    // [kKeyWarps][ROWS] m, then sums
    static constexpr int BARS = M_BUF + 2 * kKeyWarps * ROWS * 4;
    static constexpr int FLAG = BARS + 2 * NST * 8;
    static constexpr int START = FLAG + 16;                 // where the CTA's share begins
    static constexpr int BYTES = START + 64;
    static_assert(O_BUF % 16 == 0 && M_BUF % 16 == 0 && BARS % 8 == 0 && START % 8 == 0 &&
                      sizeof(Start) <= 64,
                  "alignment");
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (DT == LBV_F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7},"
            " {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7},"
            " {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DT, int D, int MT, int WM>
__global__ void __launch_bounds__(Geo<D, MT, WM>::THREADS, Geo<D, MT, WM>::CTAS)
    lbv_attend_rows_kernel(const __grid_constant__ AttendParams p,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap)
{
    using G = Geo<D, MT, WM>;
    constexpr int ROWS = G::ROWS;
    using S = Shape<ROWS, kBlock, ROWS, kExtra>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Start* start = reinterpret_cast<Start*>(smem + G::START);
    auto full = [&](int st) { return sbase + G::BARS + st * 8; };
    auto empty = [&](int st) { return sbase + G::BARS + (G::NST + st) * 8; };

    if (tid == 0) {
        for (int i = 0; i < G::NST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), G::WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (p.items && tid == 128)
        static_cast<JoinItem*>(p.items)[blockIdx.x].rows = 0;
    if (warp == 0)
        find_start<S>(p, lane, gridDim.x, kMinUnits, blockIdx.x, start);
    __syncthreads();
    if ((int)blockIdx.x >= start->ctas)
        return;
    Walk<S> w(p, *start, blockIdx.x);
    bool ok = true;

    if (warp < 4) {
        // ---- producer ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(G::REGS_PRODUCER));
        if (warp != 0)
            return;
        const int slots = min(kBlock, 1 << p.kv.page_shift);     // rows of a box
        const int boxes = kBlock / slots;                        // per 64 elements
        const int total_boxes = boxes * (D / 64) * 2;
        int n = 0;
        while (w.next()) {
            const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
            for (int b = w.b_first; b < w.b_last; ++b) {
                const int st = n % G::NST, k0 = w.key0(b);
                if (n >= G::NST && ok)
                    ok = mbar_wait(empty(st), (uint32_t)((n / G::NST - 1) & 1));
                ++n;
                if (!__all_sync(0xffffffffu, ok)) {              // a reader is stuck: no more copies
                    ok = false;
                    continue;
                }
                if (lane == 0)
                    mbar_expect_tx(full(st), G::STAGE);
                __syncwarp();
                for (int i = lane; i < total_boxes; i += 32) {
                    const int piece = i % boxes, part = i / boxes;   // part: K and V times D/64
                    const int key = k0 + piece * slots;
                    const int at = key >> p.kv.page_shift;
                    int page = -1;                               // fills zeros
                    if (key < w.x.hi && key + slots > w.x.lo)
                        page = table[at];
                    const uint32_t dst = sbase + st * G::STAGE + part * G::HALF + piece * slots * 128;
                    tma_box(dst, part < D / 64 ? &kmap : &vmap, (part % (D / 64)) * 64,
                            key & ((1 << p.kv.page_shift) - 1), w.head, page, full(st));
                }
            }
        }
        // the ring drains before shared memory goes away
        for (int i = 0; i < G::NST; ++i)
            if (n - 1 - i >= 0 && ok)
                ok = mbar_wait(empty((n - 1 - i) % G::NST), (uint32_t)(((n - 1 - i) / G::NST) & 1));
        if (!ok && lane == 0)
            atomicOr(p.status, 1u);
        return;
    }

    // ---- the rows ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(G::REGS_ROWS));
    const int ctid = tid - 128;
    const int kw = warp & (kKeyWarps - 1), wm = warp / kKeyWarps - 1;
    float* obuf = reinterpret_cast<float*>(smem + G::O_BUF);
    float* mbuf = reinterpret_cast<float*>(smem + G::M_BUF);
    float* lbuf = mbuf + kKeyWarps * ROWS;
    int* flag = reinterpret_cast<int*>(smem + G::FLAG);
    // ldmatrix lane addresses within a stage (16 keys of this warp)
    const int k_key = kw * 16 + ((lane >> 4) << 3) + (lane & 7), k_chunk = (lane >> 3) & 1;
    const int v_key = kw * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), v_chunk = lane >> 4;
    int n = 0;
    while (w.next()) {
        // Q fragments of the warp's rows, and what its rows see
        uint32_t qf[MT][D / 16][4];
        int pos[MT][2];
        uint64_t words[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = w.x.row0 + (wm * MT + mt) * 16 + h * 8 + (lane >> 2);
                const bool in = row < w.q.n * p.group;
                const int i = row / p.group, g = row - i * p.group;
                pos[mt][h] = in ? w.q.first + i : INT_MIN / 2;
                words[mt][h] = in && p.tree ? p.tree[w.q.q0 + i] : 0;
                const uint16_t* src = p.q + (int64_t)(w.q.q0 + i) * p.q_token +
                                      (int64_t)(w.head * p.group + g) * p.q_head + (lane & 3) * 2;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint16_t* a = src + ks * 16 + c * 8;
                        uint32_t v = 0;
                        if (in)
                            v = p.q_pairs ? *reinterpret_cast<const uint32_t*>(a)
                                          : (uint32_t)a[0] | ((uint32_t)a[1] << 16);
                        qf[mt][ks][c * 2 + h] = v;
                    }
            }
        float o[MT][D / 8][4];
        float m[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt][0] = m[mt][1] = -INFINITY;
            l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
                o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.f;
        }
        // keys below `open_lo` or at `open_hi` and past are hidden from some row
        const int open_hi = p.tree ? min(w.q.keys, w.q.first) : min(w.q.keys, w.q.first + w.x.row0 / p.group + 1);
        const int open_lo = p.window > 0 ? w.q.first + (w.x.row0 + w.x.rows - 1) / p.group - p.window + 1 : 0;

        for (int b = w.b_first; b < w.b_last; ++b) {
            const int st = n % G::NST, k0 = w.key0(b);
            if (ok)
                ok = mbar_wait(full(st), (uint32_t)((n / G::NST) & 1));
            ++n;
            const uint32_t ks_base = sbase + st * G::STAGE, vs_base = ks_base + (D / 64) * G::HALF;
            const int my0 = k0 + kw * 16;                        // this warp's 16 keys
            // slots past the context may hold anything: NaN times 0 is not 0
            if (my0 + 16 > w.q.keys) {
                for (int i = lane; i < 16 * (D / 8); i += 32) {
                    const int key = i / (D / 8), ch = i % (D / 8);
                    if (my0 + key >= w.q.keys)
                        *reinterpret_cast<uint4*>(smem + (vs_base - sbase) + (ch >> 3) * G::HALF +
                                                  (kw * 16 + key) * 128 + ((ch & 7) << 4)) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            float s[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s[mt][j][0] = s[mt][j][1] = s[mt][j][2] = s[mt][j][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t kf[4];
                const int ch = ks * 2 + k_chunk;
                ldsm4(ks_base + (ch >> 3) * G::HALF + k_key * 128 + (((ch & 7) ^ (k_key & 7)) << 4), kf);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma<DT>(s[mt][0], qf[mt][ks], kf[0], kf[1]);
                    mma<DT>(s[mt][1], qf[mt][ks], kf[2], kf[3]);
                }
            }
            const bool masked = my0 + 16 > open_hi || my0 < open_lo;
            bool moved = false;
            float shrink[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& t = s[mt][j][h * 2 + e];
                            t *= p.scale_log2;
                            if (masked) {
                                const int key = my0 + j * 8 + (lane & 3) * 2 + e;
                                if (!sees(p, w.q, pos[mt][h], words[mt][h], key))
                                    t = -INFINITY;
                            }
                            top = fmaxf(top, t);
                        }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    shrink[mt][h] = 1.f;
                    if (top > m[mt][h] + 8.f) {                  // also from -inf
                        shrink[mt][h] = ex2(m[mt][h] - top);
                        m[mt][h] = top;
                        moved = true;
                    }
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        l[mt][h] *= shrink[mt][h];
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[mt][j][h * 2] *= shrink[mt][h];
                            o[mt][j][h * 2 + 1] *= shrink[mt][h];
                        }
                    }
            }
            uint32_t pf[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float ref = m[mt][h] == -INFINITY ? 0.f : m[mt][h];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a = ex2(s[mt][j][h * 2] - ref), c = ex2(s[mt][j][h * 2 + 1] - ref);
                        l[mt][h] += a + c;
                        pf[mt][j * 2 + h] = pack2<DT>(a, c);
                    }
                }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
                uint32_t vf[4];
                const int ch = j * 2 + v_chunk;
                ldsm4t(vs_base + (ch >> 3) * G::HALF + v_key * 128 + (((ch & 7) ^ (v_key & 7)) << 4), vf);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma<DT>(o[mt][2 * j], pf[mt], vf[0], vf[1]);
                    mma<DT>(o[mt][2 * j + 1], pf[mt], vf[2], vf[3]);
                }
            }
            if (my0 + 16 > w.q.keys)
                fence_proxy_async_smem();                        // own stores before the next copy
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(st));
        }

        // ---- the warps' results meet ----
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[mt][h] += __shfl_xor_sync(0xffffffffu, l[mt][h], 1);
                l[mt][h] += __shfl_xor_sync(0xffffffffu, l[mt][h], 2);
                const int row = (wm * MT + mt) * 16 + h * 8 + (lane >> 2);
                if ((lane & 3) == 0) {
                    mbuf[kw * ROWS + row] = m[mt][h];
                    lbuf[kw * ROWS + row] = l[mt][h];
                }
            }
        named_bar_sync(1, G::WARPS * 32);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = (wm * MT + mt) * 16 + h * 8 + (lane >> 2);
                float top = mbuf[row];
#pragma unroll
                for (int k = 1; k < kKeyWarps; ++k)
                    top = fmaxf(top, mbuf[k * ROWS + row]);
                const float f = top == -INFINITY ? 0.f : ex2(m[mt][h] - top);
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    o[mt][j][h * 2] *= f;
                    o[mt][j][h * 2 + 1] *= f;
                }
            }
        for (int k = 0; k < kKeyWarps; ++k) {
            if (kw == k)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int row = (wm * MT + mt) * 16 + h * 8 + (lane >> 2);
                        float2* d = reinterpret_cast<float2*>(obuf + row * G::OLD + (lane & 3) * 2);
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            float2 v = make_float2(o[mt][j][h * 2], o[mt][j][h * 2 + 1]);
                            if (k > 0) {
                                const float2 a = d[j * 4];
                                v.x += a.x, v.y += a.y;
                            }
                            d[j * 4] = v;
                        }
                    }
            named_bar_sync(1, G::WARPS * 32);
        }
        // row totals (in the first warp's slots)
        const bool whole = w.whole();
        const int c0 = whole ? 0 : w.first_cta();
        const int c1 = whole ? 0 : w.last_cta();
        float* slot = p.partial + (size_t)(2 * blockIdx.x + (c0 == (int)blockIdx.x)) * G::SLOT;
        for (int i = ctid; i < w.x.rows * (D / 4); i += G::WARPS * 32) {
            const int row = i / (D / 4), d4 = i % (D / 4);
            const float4 v = *reinterpret_cast<const float4*>(obuf + row * G::OLD + d4 * 4);
            float top = mbuf[row], sum = 0.f;
#pragma unroll
            for (int k = 1; k < kKeyWarps; ++k)
                top = fmaxf(top, mbuf[k * ROWS + row]);
#pragma unroll
            for (int k = 0; k < kKeyWarps; ++k)
                sum += top == -INFINITY ? 0.f : lbuf[k * ROWS + row] * ex2(mbuf[k * ROWS + row] - top);
            if (whole) {
                finish4<DT>(p, w.q, w.head, w.x.row0 + row, d4, v, top, sum);
            } else {
                *reinterpret_cast<float4*>(slot + row * D + d4 * 4) = v;
                if (d4 == 0) {
                    slot[ROWS * D + row] = top;
                    slot[ROWS * (D + 1) + row] = sum;
                }
            }
        }
        if (!whole && p.items) {
            if (ctid == 0 && c0 == (int)blockIdx.x)
                static_cast<JoinItem*>(p.items)[c0] = {w.q.q0, w.x.row0, w.x.rows, w.head, c1 - c0 + 1};
        } else if (!whole) {
            __threadfence();
            named_bar_sync(1, G::WARPS * 32);
            if (ctid == 0)
                *flag = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
            named_bar_sync(1, G::WARPS * 32);
            if (*flag) {                                         // every part is there: join them
                __threadfence();
                join_parts<DT, D, ROWS, G::WARPS * 32>(p, w.q, w.head, w.x.row0, w.x.rows, c0, c1, ctid,
                                                       obuf, ROWS * G::OLD);
                if (ctid == 0)
                    p.counters[c0] = 0;                          // as the next call finds it
            }
        }
        named_bar_sync(1, G::WARPS * 32);                        // buffers free for the next item
    }
    if (!ok && lane == 0)
        atomicOr(p.status, 1u);
}

template <int DT, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                   cudaStream_t st)
{
    using G = Geo<D, 1, 1>;
    auto kernel = lbv_attend_rows_kernel<DT, D, 1, 1>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::BYTES);
    if (e != cudaSuccess)
        return e;
    const int ctas = sms * G::CTAS < kAttendMaxCtas ? sms * G::CTAS : kAttendMaxCtas;
    AttendParams a = p;
    const bool apart = attend_joins_apart(p, G::ROWS, ctas);
    if (!apart)
        a.items = nullptr;
    kernel<<<ctas, G::THREADS, G::BYTES, st>>>(a, kmap, vmap);
    e = cudaGetLastError();
    return e == cudaSuccess && apart ? launch_attend_join(a, (lbv_dtype)DT, G::ROWS, ctas, st) : e;
}

}  // namespace

cudaError_t launch_attend_rows(const AttendParams& p, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, lbv_dtype dt, int sms, cudaStream_t st)
{
    if (dt == LBV_F16)
        return p.kv.dim == 128 ? launch<LBV_F16, 128>(p, kmap, vmap, sms, st)
                               : launch<LBV_F16, 64>(p, kmap, vmap, sms, st);
    return p.kv.dim == 128 ? launch<LBV_BF16, 128>(p, kmap, vmap, sms, st)
                           : launch<LBV_BF16, 64>(p, kmap, vmap, sms, st);
}

size_t attend_rows_partial_floats(int dim, int sms)
{
    // two slots per CTA of the launch with the most rows times CTAs
    const int a = sms * 2 < kAttendMaxCtas ? sms * 2 : kAttendMaxCtas;
    return (size_t)2 * a * 64 * (dim + 2);
}

}  // namespace lbv

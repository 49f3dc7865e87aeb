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
//   * A producer warp copies blocks with TMA (a box is 64 elements of a head times
//     the slots of a page in the block) into a ring of 128-byte-swizzled stages, so
//     that ldmatrix reads them without bank conflicts.
//   * Four warps share a block: each takes the scores of 16 keys (mma.sync
//     m16n8k16 with the rows as M), they agree on the rows' references, exchange
//     their probabilities through shared memory, and each adds up a quarter of the
//     head's elements over all 64 keys.  So no sums have to be joined at an item's
//     end, and the accumulators take a quarter of the registers.  One tile of 16
//     rows a read of the keys is what mma.sync sustains beside memory: it takes
//     about 32 cycles an instruction and SM quarter, and tiles of 32 rows ran 1.4
//     times slower than memory (310 us for 64 requests of one token, 220 with 16
//     rows).  Larger tiles go to the tensor-memory kernel (attend_tiles.cu).
//
// 64 requests of one token over 500 to 16,384 keys, 48 query over 8 key/value heads of
// 128: 216 to 220 us with the join, 6.4 to 6.5 TB/s, 94 to 96 % of what a copy reaches.  One request over
// 2,011 keys: 9.5 us, of round trips to memory.  32 requests of 1 to 8 tokens, 32 query
// over 8 heads of 64, window 4096: 50 us, 61 %; a third of them has two row tiles, which
// read their keys twice (60 us by the tensor-memory kernel).
#include "attend_common.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kBlock = 64;                       // keys per block
constexpr int kKeyWarps = 4;
// Units of an item beside its blocks, and the least share of a CTA (below, joining
// costs more than it saves).
constexpr int kExtra = 3, kMinUnits = 2;

template <int D>
struct Geo {
    static constexpr int ROWS = 16;
    static constexpr int THREADS = kKeyWarps * 32 + 32;     // and the producer
    static constexpr int HALF = kBlock * 128;               // 64 elements of 64 keys
    static constexpr int STAGE = 2 * (D / 64) * HALF;       // K then V
    // CTAs on an SM, which share about 192 KB of ring: a block of small heads is
    // short, and more of them have to be under way
    static constexpr int CTAS = D == 64 ? 4 : 2;
    static constexpr int NST = 196608 / CTAS / STAGE;
    static constexpr int SLOT = ROWS * (D + 3);             // floats of one partial result
    static constexpr int PLD = kBlock * 2 + 16;             // bytes of a row of probabilities
    // shared memory; from the probabilities to the barriers it is also the join's
    // scratch, which takes 2 floats a part for one row at least
    static constexpr int P_BUF = NST * STAGE;
    static constexpr int Q_BUF = P_BUF + ROWS * PLD + 16;   // the item's queries
    static constexpr int QLD = D * 2 + 16;                  // bytes of a row of them
    static constexpr int M_BUF = Q_BUF + ROWS * QLD;        // [kKeyWarps][ROWS] block maxima; sums, twice
    static constexpr int BARS = M_BUF + 2 * kKeyWarps * ROWS * 4;
    static constexpr int FLAG = BARS + 2 * NST * 8;
    static constexpr int START = FLAG + 16;                 // where the CTA's share begins
    static constexpr int BYTES = START + 64;
    static_assert(P_BUF % 16 == 0 && Q_BUF % 16 == 0 && M_BUF % 16 == 0 && BARS % 8 == 0 &&
                      START % 8 == 0 && sizeof(Start) <= 64 && (BARS - P_BUF) / 4 >= 2 * kAttendMaxCtas + 3,
                  "layout");
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

template <int DT, int D>
__global__ void __launch_bounds__(Geo<D>::THREADS, Geo<D>::CTAS)
    lbv_attend_rows_kernel(const __grid_constant__ AttendParams p,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap)
{
    using G = Geo<D>;
    constexpr int ROWS = G::ROWS;
    using S = Shape<ROWS, kBlock, kExtra>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Start* start = reinterpret_cast<Start*>(smem + G::START);
    auto full = [&](int st) { return sbase + G::BARS + st * 8; };
    auto empty = [&](int st) { return sbase + G::BARS + (G::NST + st) * 8; };

    if (tid == 0) {
        for (int i = 0; i < G::NST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kKeyWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    after_previous();
    if (p.items && tid == 0)
        static_cast<JoinItem*>(p.items)[blockIdx.x].rows = 0;
    if (warp == 0)
        find_start<S>(p, lane, gridDim.x, kMinUnits, blockIdx.x, start);
    __syncthreads();
    if ((int)blockIdx.x >= start->ctas)
        return;
    Walk<S> w(p, *start, blockIdx.x);
    bool ok = true;

    if (warp == kKeyWarps) {
        // ---- producer ----
        const int slots = min(kBlock, 1 << p.kv.page_shift);     // rows of a box
        const int boxes = kBlock / slots;                        // per 64 elements
        const int total_boxes = boxes * (D / 64) * 2;
        int n = 0;                                               // blocks asked for
        while (ok && w.next()) {
            const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
            for (int b = w.b_first; b < w.b_last; ++b) {
                const int st = n % G::NST, k0 = w.key0(b);
                // A stage is asked for again when it has been read, and its last copies have
                // landed (readers that gave up free it all the same).
                if (n >= G::NST) {
                    const uint32_t parity = (uint32_t)((n / G::NST - 1) & 1);
                    ok = mbar_wait(empty(st), parity, p.wait_limit) && mbar_wait(full(st), parity, p.wait_limit);
                }
                ok = __all_sync(0xffffffffu, ok && ((unsigned)n < p.first_copies || blockIdx.x > 0));
                if (!ok)                                         // no more copies
                    break;
                ++n;
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
        // the copies land before shared memory goes away, also after a wait that ran out
        for (int i = 0; i < G::NST; ++i)
            if (n - 1 - i >= 0 && !mbar_wait(full((n - 1 - i) % G::NST), (uint32_t)(((n - 1 - i) / G::NST) & 1),
                                             p.wait_limit))
                ok = false;
        if (!ok && lane == 0)
            atomicOr(p.status, 1u);
        return;
    }

    // ---- the rows ----
    constexpr int TEAM = kKeyWarps * 32;                         // threads beside the producer
    unsigned char* pbuf = smem + G::P_BUF;
    float* tops = reinterpret_cast<float*>(smem + G::M_BUF);
    int* flag = reinterpret_cast<int*>(smem + G::FLAG);
    const int r0 = lane >> 2;                                    // the thread's rows: r0 and r0 + 8
    // ldmatrix lane addresses: 16 keys of this warp in K, 16 keys of a step in V, the
    // rows of a step in P and Q
    const int k_key = warp * 16 + ((lane >> 4) << 3) + (lane & 7), k_chunk = (lane >> 3) & 1;
    const int v_key = (((lane >> 3) & 1) << 3) + (lane & 7), v_chunk = warp * (D / 32) + (lane >> 4);
    const uint32_t p_lane = sbase + G::P_BUF + (lane & 15) * G::PLD + (lane >> 4) * 16;
    const uint32_t q_lane = sbase + G::Q_BUF + (lane & 15) * G::QLD + (lane >> 4) * 16;
    constexpr int NT = D / 32;                                   // 8-element tiles of this warp's quarter
    int n = 0;
    while (w.next()) {
        // the queries by way of shared memory, and what the rows see
        for (int i = tid; i < ROWS * (D / 8); i += TEAM) {
            const int r = i / (D / 8), ch = i % (D / 8), row = w.x.row0 + r;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < w.x.rows) {
                const int t = token_of(p, row);
                const uint16_t* src = p.q + (int64_t)(w.q.q0 + t) * p.q_token +
                                      (int64_t)(w.head * p.group + row - t * p.group) * p.q_head + ch * 8;
                if (p.q_wide) {
                    v = __ldg(reinterpret_cast<const uint4*>(src));
                } else {
                    uint32_t e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        e[k] = (uint32_t)src[2 * k] | ((uint32_t)src[2 * k + 1] << 16);
                    v = make_uint4(e[0], e[1], e[2], e[3]);
                }
            }
            *reinterpret_cast<uint4*>(smem + G::Q_BUF + r * G::QLD + ch * 16) = v;
        }
        int pos[2];
        uint64_t words[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool in = r0 + h * 8 < w.x.rows;
            const int i = token_of(p, w.x.row0 + r0 + h * 8);
            pos[h] = in ? w.q.first + i : INT_MIN / 2;
            words[h] = in && p.tree ? p.tree[w.q.q0 + i] : 0;
        }
        named_bar_sync(1, TEAM);
        uint32_t qf[D / 16][4];
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
            ldsm4(q_lane + ks * 32, qf[ks]);
        float o[NT][4];
        float m[2] = {-INFINITY, -INFINITY};
        float l[2] = {0.f, 0.f}, x[2] = {0.f, 0.f};  // sums of rounded, of exact probabilities
#pragma unroll
        for (int j = 0; j < NT; ++j)
            o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        // keys below `open_lo` or at `open_hi` and past are hidden from some row
        const int open_hi = p.tree ? min(w.q.keys, w.q.first)
                                   : min(w.q.keys, w.q.first + token_of(p, w.x.row0) + 1);
        const int open_lo =
            p.window > 0 ? w.q.first + token_of(p, w.x.row0 + w.x.rows - 1) - p.window + 1 : 0;

        for (int b = w.b_first; b < w.b_last; ++b) {
            const int st = n % G::NST, k0 = w.key0(b);
            if (ok)
                ok = mbar_wait(full(st), (uint32_t)((n / G::NST) & 1), p.wait_limit);
            ++n;
            const uint32_t ks_base = sbase + st * G::STAGE, vs_base = ks_base + (D / 64) * G::HALF;
            const int my0 = k0 + warp * 16;                      // this warp's 16 keys
            // slots past the context may hold anything: NaN times 0 is not 0 (the other
            // warps read V after the barriers below)
            const bool tail = k0 + kBlock > w.q.keys;
            if (tail)
                for (int i = lane; i < 16 * (D / 8); i += 32) {
                    const int key = i / (D / 8), ch = i % (D / 8);
                    if (my0 + key >= w.q.keys)
                        *reinterpret_cast<uint4*>(smem + (vs_base - sbase) + (ch >> 3) * G::HALF +
                                                  (warp * 16 + key) * 128 + ((ch & 7) << 4)) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
            float s[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t kf[4];
                const int ch = ks * 2 + k_chunk;
                ldsm4(ks_base + (ch >> 3) * G::HALF + k_key * 128 + (((ch & 7) ^ (k_key & 7)) << 4), kf);
                mma<DT>(s[0], qf[ks], kf[0], kf[1]);
                mma<DT>(s[1], qf[ks], kf[2], kf[3]);
            }
            const bool masked = my0 + 16 > open_hi || my0 < open_lo;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& t = s[j][h * 2 + e];
                        t *= p.scale_log2;
                        if (masked && !sees(p, w.q, pos[h], words[h], my0 + j * 8 + (lane & 3) * 2 + e))
                            t = -INFINITY;
                        top = fmaxf(top, t);
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if ((lane & 3) == 0)
                    tops[warp * ROWS + h * 8 + r0] = top;
            }
            named_bar_sync(1, TEAM);
            // the block's maxima, the same for every warp
            bool moved = false;
            float shrink[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* t = tops + h * 8 + r0;
                const float top = fmaxf(fmaxf(t[0], t[ROWS]), fmaxf(t[2 * ROWS], t[3 * ROWS]));
                shrink[h] = 1.f;
                if (top > m[h] + 8.f) {                          // also from -inf
                    shrink[h] = ex2(m[h] - top);
                    m[h] = top;
                    moved = true;
                }
                const float ref = m[h] == -INFINITY ? 0.f : m[h];
                l[h] *= shrink[h];
                x[h] *= shrink[h];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float a = ex2(s[j][h * 2] - ref), c = ex2(s[j][h * 2 + 1] - ref);
                    const uint32_t r = pack2<DT>(a, c);
                    const float2 v = unpack2<DT>(r);
                    x[h] += a + c;                               // of this warp's keys
                    l[h] += v.x + v.y;
                    *reinterpret_cast<uint32_t*>(pbuf + (h * 8 + r0) * G::PLD +
                                                 (warp * 16 + j * 8 + (lane & 3) * 2) * 2) = r;
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[j][0] *= shrink[0], o[j][1] *= shrink[0];
                    o[j][2] *= shrink[1], o[j][3] *= shrink[1];
                }
            }
            named_bar_sync(1, TEAM);
#pragma unroll
            for (int ks = 0; ks < kBlock / 16; ++ks) {
                uint32_t pf[4];
                ldsm4(p_lane + ks * 32, pf);
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    uint32_t vf[4];
                    const int ch = j * 2 + v_chunk, key = ks * 16 + v_key;
                    ldsm4t(vs_base + (ch >> 3) * G::HALF + key * 128 + (((ch & 7) ^ (key & 7)) << 4), vf);
                    mma<DT>(o[2 * j], pf, vf[0], vf[1]);
                    mma<DT>(o[2 * j + 1], pf, vf[2], vf[3]);
                }
            }
            if (tail)
                fence_proxy_async_smem();                        // own stores before the next copy
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(st));
        }

        // ---- the item's result: each warp has a quarter of the elements ----
        named_bar_sync(1, TEAM);                                 // the last maxima have been read
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            x[h] += __shfl_xor_sync(0xffffffffu, x[h], 1);
            x[h] += __shfl_xor_sync(0xffffffffu, x[h], 2);
            if ((lane & 3) == 0) {
                tops[warp * ROWS + h * 8 + r0] = l[h];
                tops[(kKeyWarps + warp) * ROWS + h * 8 + r0] = x[h];
            }
        }
        named_bar_sync(1, TEAM);
        const bool whole = w.whole();
        const int c0 = whole ? 0 : w.first_cta();
        const int c1 = whole ? 0 : w.last_cta();
        float* slot = p.partial + (size_t)(2 * blockIdx.x + (c0 == (int)blockIdx.x)) * G::SLOT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = h * 8 + r0, row = w.x.row0 + r;
            if (r >= w.x.rows)
                continue;
            const float* t = tops + r;
            const float sum = (t[0] + t[ROWS]) + (t[2 * ROWS] + t[3 * ROWS]);
            const float exact = (t[4 * ROWS] + t[5 * ROWS]) + (t[6 * ROWS] + t[7 * ROWS]);
            const int i = token_of(p, row), head = w.head * p.group + row - i * p.group;
            const int64_t tok = w.q.q0 + i;
            const bool first = warp == 0 && (lane & 3) == 0;
            const int e0 = warp * (D / 4) + (lane & 3) * 2;
            if (whole) {
                const float f = 1.f / sum;
                uint16_t* d = p.out + tok * p.out_token + (int64_t)head * p.out_head + e0;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t v = sum == 0.f ? 0u : pack2<DT>(o[j][h * 2] * f, o[j][h * 2 + 1] * f);
                    store_row<2>(d + j * 8, &v);
                }
                if (p.lse && first)
                    p.lse[tok * p.heads + head] = lse_of(m[h], exact);
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    *reinterpret_cast<float2*>(slot + r * D + e0 + j * 8) =
                        make_float2(o[j][h * 2], o[j][h * 2 + 1]);
                if (first) {
                    slot[ROWS * D + r] = m[h];
                    slot[ROWS * (D + 1) + r] = sum;
                    slot[ROWS * (D + 2) + r] = exact;
                }
            }
        }
        if (!whole && p.items) {
            if (tid == 0 && c0 == (int)blockIdx.x)
                static_cast<JoinItem*>(p.items)[c0] = {w.q.q0, w.x.row0, w.x.rows, w.head, c1 - c0 + 1};
        } else if (!whole) {
            __threadfence();
            named_bar_sync(1, TEAM);
            if (tid == 0)
                *flag = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
            named_bar_sync(1, TEAM);
            if (*flag) {                                         // every part is there: join them
                __threadfence();
                join_parts<DT, D, ROWS, TEAM>(p, w.q, w.head, w.x.row0, w.x.rows, c0, c1, tid,
                                              reinterpret_cast<float*>(pbuf), (G::BARS - G::P_BUF) / 4);
                if (tid == 0)
                    p.counters[c0] = 0;                          // as the next call finds it
            }
            named_bar_sync(1, TEAM);                             // the flag has been read
        }
    }
    if (!ok && lane == 0)
        atomicOr(p.status, 1u);
}

template <int DT, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                   cudaStream_t st)
{
    using G = Geo<D>;
    auto kernel = lbv_attend_rows_kernel<DT, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::BYTES);
    if (e != cudaSuccess)
        return e;
    const int ctas = sms * G::CTAS < kAttendMaxCtas ? sms * G::CTAS : kAttendMaxCtas;
    AttendParams a = p;
    const bool apart = attend_joins_apart(p, G::ROWS, ctas);
    if (!apart)
        a.items = nullptr;
    e = launch_after(kernel, dim3((unsigned)ctas), G::THREADS, G::BYTES, st, a, kmap, vmap);
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
    // two slots per CTA
    const int ctas = sms * (dim == 64 ? Geo<64>::CTAS : Geo<128>::CTAS);
    const int a = ctas < kAttendMaxCtas ? ctas : kAttendMaxCtas;
    return (size_t)2 * a * 16 * (dim + 3);
}

}  // namespace lbv

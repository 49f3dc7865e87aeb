// attend4_rows.cu -- attention of few new tokens over a paged cache of 4 bits (plain
// decoding, verify calls, trees of drafted tokens).
//
// The sums of attend_rows.cu.  A quarter of the bytes leaves a quarter of the time for
// everything else, so the products are turned around: keys are the 128 rows of the
// tensor core's tile and the queries, a few, its columns,
//     S^T = K Q^T (128 keys x N rows),   O^T += V^T P^T (D x N rows).
// An MMA's time then goes by its operands' bytes, not by padded rows, and
//   * the scores of a key are a thread's: the thread that loads and expands a key's
//     codes (32 bytes a load) writes the key to tensor memory, where the first product
//     takes it from, without a detour by shared memory; it gets the key's scores from
//     there, masks them, takes the exponentials, and adds them up for itself, one sum
//     a row, joined with the other keys' at the item's end;
//   * it writes its key's values and probabilities to shared memory as a row each, which
//     are the second product's operands as they are: rows along the contracted dimension.
// A group of four warps does this block by block for a share of its own; the groups of a
// CTA have nothing to do with one another but the SM, whose schedulers take one's
// arithmetic while another waits.  Shares, items and references are those of attend_common.cuh
// (a reference moves when a score passes it by more than 8); the parts of divided items
// are added by a launch of their own (attend_join.cu).
//
// The divisor adds the probabilities before their rounding to 16 bits (off by 2^-9 of a
// value for a row that one key dominates; the values themselves are held to 2^-5).
#include <algorithm>

#include "attend_common.cuh"
#include "attend_tc.cuh"
#include "kv4.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kKeys = 128;                       // keys per block, one a thread
// Units of a block and of an item beside its blocks; the least share of a group.
constexpr int kBlockUnits = 4, kExtra = 6, kMinUnits = 4;

// N: rows of an item, 16 or 48.
template <int D, int N>
struct Geo4 {
    // groups of four warps: as many as shared memory has room for
    static constexpr int GROUPS = N == 16 ? 4 : 3;
    static constexpr int THREADS = GROUPS * 128;
    static constexpr int HALF = kKeys * 128;                // 64 elements of 128 keys
    // a group's shared memory: V; P, whose rows have room for 64; Q; what the rows need
    static constexpr int V = 0;
    static constexpr int P = D / 64 * HALF;
    static constexpr int Q = P + HALF;
    static constexpr int QHALF = N * 128;
    static constexpr int INFO = Q + D / 64 * QHALF;
    static constexpr int WORDS = INFO;                      // uint64 [N]: the rows' words of the tree
    static constexpr int POS = WORDS + 8 * N;               // int [N]: their positions
    static constexpr int REF = POS + 4 * N;                 // float [N]: references
    static constexpr int LIMIT = REF + 4 * N;               // what a score passes to move them
    static constexpr int MINUS = LIMIT + 4 * N;             // what is added to a score
    static constexpr int FACTOR = MINUS + 4 * N;            // of the sums, when they move
    static constexpr int PARTS = FACTOR + 4 * N;            // [4][N]: warps' maxima and sums
    static constexpr int BARS = PARTS + 16 * N;
    static constexpr int START = BARS + 16;
    static constexpr int SIZE = (START + 64 + 1023) / 1024 * 1024;
    static constexpr int TMEM = GROUPS * SIZE;              // tensor-memory address
    static constexpr int BYTES = TMEM + 16;
    // a group's tensor memory columns
    static constexpr uint32_t K_COL = 0, S_COL = D / 2, O_COL = S_COL + N, COLUMNS = O_COL + N;
    static constexpr int SLOT = N * (D + 3);                // floats of one partial result
    static_assert(INFO % 16 == 0 && BARS % 8 == 0 && START % 8 == 0 && sizeof(Start) <= 64, "layout");
    static_assert(BYTES <= 227 * 1024 && GROUPS * COLUMNS <= 512 && N <= 64, "room");
};

// Whether any of the group's threads says so; all of them meet here.
__device__ __forceinline__ bool any_of_group(int bar, bool mine)
{
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %2, 0;\n bar.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any)
        : "r"(bar), "r"((uint32_t)mine)
        : "memory");
    return any != 0;
}

// The largest of a warp's 32 values.
__device__ __forceinline__ float warp_max(float x)
{
    int b = __float_as_int(x);
    b ^= (b >> 31) & 0x7FFFFFFF;                 // ordered as the floats are
    b = __reduce_max_sync(0xffffffffu, b);
    return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF));
}

template <int DT, int D, int N>
__global__ void __launch_bounds__(Geo4<D, N>::THREADS, 1)
    lbv_attend4_rows_kernel(const __grid_constant__ AttendParams p)
{
    using G = Geo4<D, N>;
    using S = Shape<N, kKeys, kExtra, kBlockUnits>;
    constexpr int CH = N / 16;                                   // chunks of 16 rows
    extern __shared__ __align__(1024) unsigned char smem_all[];
    const int tid = threadIdx.x, group = tid >> 7, row = tid & 127, warp = (tid >> 5) & 3, lane = tid & 31;
    unsigned char* smem = smem_all + group * G::SIZE;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t s_full = sbase + G::BARS, o_done = s_full + 8;
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem_all + G::TMEM);
    Start* start = reinterpret_cast<Start*>(smem + G::START);
    // shares go to the SMs first, then to their groups
    const int share = group * gridDim.x + blockIdx.x;
    const int bar = 1 + group;

    if (row == 0) {
        mbar_init(s_full, 1);
        mbar_init(o_done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid < 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        tc_fence_before();
    }
    after_previous();
    if (row == 0)
        static_cast<JoinItem*>(p.items)[share].rows = 0;
    if (warp == 0)
        find_start<S>(p, lane, gridDim.x * G::GROUPS, kMinUnits, share, start);
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_slot, 0) + group * G::COLUMNS;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t k_at = tm + lanes + G::K_COL, s_at = tm + lanes + G::S_COL, o_at = tm + lanes + G::O_COL;
    bool ok = true;

    if (share < start->ctas) {
        uint64_t* words = reinterpret_cast<uint64_t*>(smem + G::WORDS);
        int* pos = reinterpret_cast<int*>(smem + G::POS);
        float* ref = reinterpret_cast<float*>(smem + G::REF);
        float* limit = reinterpret_cast<float*>(smem + G::LIMIT);
        float* minus = reinterpret_cast<float*>(smem + G::MINUS);
        float* factor = reinterpret_cast<float*>(smem + G::FACTOR);
        float* parts = reinterpret_cast<float*>(smem + G::PARTS);
        const int cs = kv4::chunk_shift(p.kv), slot_mask = (1 << p.kv.page_shift) - 1, chunk_mask = (1 << cs) - 1;
        // scores are c times the products; a scale of zero clears Q
        const float c = p.scale_log2 == 0.f ? 1.f : p.scale_log2;
        const float hidden = c < 0.f ? INFINITY : -INFINITY;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok)
                ok = mbar_wait(b, parity, p.wait_limit);
        };
        Walk<S> w(p, *start, share);
        int n = 0;                                               // blocks so far
        while (w.next()) {
            const int rows = w.x.rows, nb = w.b_last - w.b_first;
            const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
            // this thread's key of block j of the share, its page (-1: zeros) and its chunk
            auto key_of = [&](int j) { return w.key0(w.b_first + j) + row; };
            auto page_of = [&](int j) {
                const int key = key_of(j);
                return j < nb && wanted(p, w.x.lo, w.x.hi, key, 1) ? table[key >> p.kv.page_shift] : -1;
            };
            auto chunk_of = [&](int page, int j) -> const uint8_t* {
                return page < 0 || page >= p.kv.pages ? nullptr
                                                      : kv4::chunk(p.kv, page, w.head, key_of(j) & slot_mask);
            };
            kv4::Held<D> k, v;
            int page1;                                           // of the next block
            {
                const int page0 = page_of(0);
                page1 = page_of(1);
                const uint8_t* at = chunk_of(page0, 0);
                const int s = key_of(0) & chunk_mask;
                k.load(at, 0, s, cs);
                v.load(at, 1, s, cs);
            }
            // the queries, and what the rows see
            for (int i = row; i < rows * (D / 8); i += 128) {
                const int r = i / (D / 8), ch = i % (D / 8), qrow = w.x.row0 + r;
                const int t = token_of(p, qrow);
                const uint16_t* src = p.q + (int64_t)(w.q.q0 + t) * p.q_token +
                                      (int64_t)(w.head * p.group + qrow - t * p.group) * p.q_head + ch * 8;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (p.scale_log2 == 0.f) {
                } else if (p.q_wide) {
                    x = __ldg(reinterpret_cast<const uint4*>(src));
                } else {
                    uint32_t e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        e[j] = (uint32_t)src[2 * j] | ((uint32_t)src[2 * j + 1] << 16);
                    x = make_uint4(e[0], e[1], e[2], e[3]);
                }
                *reinterpret_cast<uint4*>(smem + G::Q + (ch >> 3) * G::QHALF + r * 128 +
                                          (((ch & 7) ^ (r & 7)) << 4)) = x;
            }
            fence_proxy_async_smem();
            if (row < N) {
                const int i = token_of(p, w.x.row0 + row);
                pos[row] = row < rows ? w.q.first + i : INT_MIN / 2;
                words[row] = row < rows && p.tree ? p.tree[w.q.q0 + i] : 0;
                ref[row] = limit[row] = -INFINITY;
                minus[row] = 0.f;
            }
            float x[N];                                          // this key's share of the rows' sums
#pragma unroll
            for (int r = 0; r < N; ++r)
                x[r] = 0.f;
            // keys below `open_lo` or at `open_hi` and past are hidden from some row
            const int open_hi = p.tree ? min(w.q.keys, w.q.first)
                                       : min(w.q.keys, w.q.first + token_of(p, w.x.row0) + 1);
            const int open_lo =
                p.window > 0 ? w.q.first + token_of(p, w.x.row0 + rows - 1) - p.window + 1 : 0;

            for (int j = 0; j < nb; ++j, ++n) {
                const int key = key_of(j), page2 = page_of(j + 2);
                const bool masked = key - row + kKeys > open_hi || key - row < open_lo;
                const uint8_t* next = chunk_of(page1, j + 1);
                const int next_s = key_of(j + 1) & chunk_mask;
                page1 = page2;
                // ---- the key ----
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    const uint32_t sc = kv4::both_scales(k.scales[part]), bi = kv4::both_biases(k.scales[part]);
                    uint32_t e[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        kv4::expand<DT>(k.codes[part][i], sc, bi, reinterpret_cast<uint32_t(&)[4]>(e[4 * i]));
                    tmem_st32(k_at + part * 32, e);
                }
                k.load(next, 0, next_s, cs);
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(bar, 128);
                // (the test of the bounded waits leaves the product out)
                if (warp == 0 && ((unsigned)n < p.first_copies || share > 0)) {
                    tc_fence_after();
                    const uint64_t b = desc128(sbase + G::Q, 0);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        mma4_tk(tm + G::S_COL, tm + G::K_COL + h * 32, b + h * (G::QHALF >> 4), idesc<DT>(N, false),
                                h > 0);
                    commit(s_full);
                }
                // ---- the value, when the last block's has been used ----
                if (n > 0)
                    wait(o_done, (uint32_t)((n - 1) & 1));
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    const uint32_t sc = kv4::both_scales(v.scales[part]), bi = kv4::both_biases(v.scales[part]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t e[4];
                        kv4::expand<DT>(v.codes[part][i], sc, bi, e);
                        *reinterpret_cast<uint4*>(smem + G::V + part * G::HALF + row * 128 + ((i ^ (row & 7)) << 4)) =
                            make_uint4(e[0], e[1], e[2], e[3]);
                    }
                }
                v.load(next, 1, next_s, cs);
                // ---- the key's scores, 16 rows at a time ----
                wait(s_full, (uint32_t)(n & 1));
                tc_fence_after();
                float t[16];
                auto scores = [&](int ch) {
                    tmem_ld16(s_at + ch * 16, t);
                    tmem_wait_ld();
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (!sees(p, w.q, pos[ch * 16 + i], words[ch * 16 + i], key))
                                t[i] = hidden;
                    }
                };
                bool over = false;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
                    if (ch * 16 < rows) {
                        scores(ch);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            over = over || (ch * 16 + i < rows && t[i] * c > limit[ch * 16 + i]);
                    }
                if (any_of_group(bar, over)) {
                    // some reference moves: the block's maxima
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch)
                        if (ch * 16 < rows) {
                            if (CH > 1)
                                scores(ch);
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float top = warp_max(t[i] * c);
                                if (lane == 0)
                                    parts[warp * N + ch * 16 + i] = top;
                            }
                        }
                    named_bar_sync(bar, 128);
                    if (row < rows) {
                        const float* q = parts + row;
                        const float top = fmaxf(fmaxf(q[0], q[N]), fmaxf(q[2 * N], q[3 * N]));
                        float f = 1.f;
                        if (top > limit[row]) {                  // also from -inf
                            f = ex2(ref[row] - top);
                            ref[row] = top;
                            limit[row] = top + 8.f;
                            minus[row] = -top;
                        }
                        factor[row] = f;
                    }
                    named_bar_sync(bar, 128);
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch)
                        if (ch * 16 < rows) {
                            float o[16];
                            if (j > 0) {
                                tmem_ld16(o_at + ch * 16, o);
                                tmem_wait_ld();
                            }
                            uint32_t r[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float f = ch * 16 + i < rows ? factor[ch * 16 + i] : 1.f;
                                x[ch * 16 + i] *= f;
                                r[i] = __float_as_uint(o[i] * f);
                            }
                            if (j > 0)
                                tmem_st16(o_at + ch * 16, r);
                        }
                    tmem_wait_st();
                }
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
                    if (ch * 16 < rows) {
                        if (CH > 1)
                            scores(ch);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (ch * 16 + h * 8 < rows) {
                                uint32_t r[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const int at = h * 8 + 2 * i;
                                    const float a = ex2(fmaf(t[at], c, minus[ch * 16 + at]));
                                    const float b = ex2(fmaf(t[at + 1], c, minus[ch * 16 + at + 1]));
                                    x[ch * 16 + at] += a;
                                    x[ch * 16 + at + 1] += b;
                                    r[i] = pack2<DT>(a, b);
                                }
                                *reinterpret_cast<uint4*>(smem + G::P + row * 128 + (((ch * 2 + h) ^ (row & 7)) << 4)) =
                                    make_uint4(r[0], r[1], r[2], r[3]);
                            }
                    }
                fence_proxy_async_smem();
                tc_fence_before();
                named_bar_sync(bar, 128);
                if (warp == 0) {
                    tc_fence_after();
                    // (heads of 64 elements: the rows past them are P's, and not used)
                    const uint64_t a = desc128(sbase + G::V, G::HALF), b = desc128(sbase + G::P, G::HALF);
#pragma unroll
                    for (int h = 0; h < 2; ++h)                  // 64 keys at a time
                        mma4_rr(tm + G::O_COL, a + h * 512, b + h * 512, idesc<DT>(N, true, true), j > 0 || h > 0);
                    commit(o_done);
                }
            }

            // ---- the item's result: a thread has an element of every row ----
#pragma unroll
            for (int r = 0; r < N; ++r)
                if (r < rows) {
                    float s = x[r];
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1)
                        s += __shfl_xor_sync(0xffffffffu, s, d);
                    if (lane == 0)
                        parts[warp * N + r] = s;
                }
            named_bar_sync(bar, 128);
            wait(o_done, (uint32_t)((n - 1) & 1));
            tc_fence_after();
            const bool whole = w.whole();
            const int c0 = whole ? 0 : w.first_cta(), c1 = whole ? 0 : w.last_cta();
            float* slot = p.partial + (size_t)(2 * share + (c0 == share)) * G::SLOT;
            auto sum_of = [&](int r) { return (parts[r] + parts[N + r]) + (parts[2 * N + r] + parts[3 * N + r]); };
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
                if (ch * 16 < rows) {
                    float o[16];
                    tmem_ld16(o_at + ch * 16, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int r = ch * 16 + i;
                        if (r < rows && row < D) {
                            if (whole) {
                                const int qrow = w.x.row0 + r, tok = token_of(p, qrow);
                                const float s = sum_of(r);
                                const uint32_t y = s > 0.f ? pack2<DT>(o[i] / s, 0.f) : 0u;
                                p.out[(int64_t)(w.q.q0 + tok) * p.out_token +
                                      (int64_t)(w.head * p.group + qrow - tok * p.group) * p.out_head + row] =
                                    (uint16_t)y;
                            } else {
                                slot[r * D + row] = o[i];
                            }
                        }
                    }
                }
            if (row < rows) {
                const float s = sum_of(row);
                if (!whole) {
                    slot[N * D + row] = ref[row];
                    slot[N * (D + 1) + row] = slot[N * (D + 2) + row] = s;
                } else if (p.lse) {
                    const int qrow = w.x.row0 + row, tok = token_of(p, qrow);
                    p.lse[(int64_t)(w.q.q0 + tok) * p.heads + w.head * p.group + qrow - tok * p.group] =
                        lse_of(ref[row], s);
                }
            }
            if (!whole && row == 0 && c0 == share)
                static_cast<JoinItem*>(p.items)[c0] = {w.q.q0, w.x.row0, rows, w.head, c1 - c0 + 1};
            tc_fence_before();
            named_bar_sync(bar, 128);                            // what the rows need has been read
        }
        // the last product ends before tensor memory goes away, also after a wait that ran out
        if (n > 0 && !mbar_wait(o_done, (uint32_t)((n - 1) & 1), p.wait_limit))
            ok = false;
        if (!ok)
            atomicOr(p.status, 1u);
    }
    __syncthreads();
    if (tid < 32) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem_slot) : "memory");
    }
}

template <int DT, int D, int N>
cudaError_t launch(const AttendParams& p, int sms, cudaStream_t st)
{
    using G = Geo4<D, N>;
    auto kernel = lbv_attend4_rows_kernel<DT, D, N>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::BYTES);
    if (e != cudaSuccess)
        return e;
    const int ctas = std::min(sms, kAttendMaxCtas / G::GROUPS);
    e = launch_after(kernel, dim3((unsigned)ctas), G::THREADS, G::BYTES, st, p);
    return e == cudaSuccess ? launch_attend_join(p, (lbv_dtype)DT, N, ctas * G::GROUPS, st) : e;
}

template <int DT, int D>
cudaError_t launch_rows(const AttendParams& p, int sms, cudaStream_t st)
{
    return attend_average_rows(p) <= 16 ? launch<DT, D, 16>(p, sms, st) : launch<DT, D, 48>(p, sms, st);
}

}  // namespace

cudaError_t launch_attend4_rows(const AttendParams& p, const CUtensorMap&, const CUtensorMap&, lbv_dtype dt, int sms,
                                cudaStream_t st)
{
    if (dt == LBV_F16)
        return p.kv.dim == 128 ? launch_rows<LBV_F16, 128>(p, sms, st) : launch_rows<LBV_F16, 64>(p, sms, st);
    return p.kv.dim == 128 ? launch_rows<LBV_BF16, 128>(p, sms, st) : launch_rows<LBV_BF16, 64>(p, sms, st);
}

size_t attend4_rows_partial_floats(int dim, int sms)
{
    // two slots a group: three groups of 48 rows, more than four of 16
    return (size_t)2 * std::min(3 * sms, kAttendMaxCtas) * 48 * (dim + 3);
}

}  // namespace lbv

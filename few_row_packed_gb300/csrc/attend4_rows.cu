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
// A reference that every score passes, negated: nothing has been seen yet.
constexpr float kNone = 1e30f;

// N: rows of an item, 16 or 48.
template <int D, int N>
struct Geo4 {
    // groups of four warps, and stages of values as they are held: what shared memory has room for
    static constexpr int GROUPS = D == 64 && N == 16 ? 4 : 3;
    static constexpr int VST = N == 16 ? 2 : 1;
    static constexpr int THREADS = GROUPS * 128;
    static constexpr int HALF = kKeys * 128;                // 64 elements of 128 keys
    // a group's operands: V in rows of 128 bytes, P in rows of 16 probabilities, Q
    static constexpr int V = 0;
    static constexpr int P = D / 64 * HALF;
    static constexpr int PCHUNK = kKeys * 32;
    static constexpr int Q = P + N / 16 * PCHUNK;
    static constexpr int QHALF = N * 128;
    static constexpr int SIZE = Q + D / 64 * QHALF;
    // behind the groups' operands, what else each has: a block's keys and values as they are
    // held (codes, then scales), and what the rows need
    static constexpr int CODES = kKeys * 32 * (D / 64), HELD = kKeys * 36 * (D / 64);
    static constexpr int KHELD = 0;
    static constexpr int VHELD = HELD;
    static constexpr int WORDS = VHELD + VST * HELD;        // uint64 [N]: the rows' words of the tree
    static constexpr int POS = WORDS + 8 * N;               // int [N]: their positions
    static constexpr int MINUS = POS + 4 * N;               // float [N]: their references, negated
    static constexpr int PARTS = MINUS + 4 * N;             // [4][N]: warps' maxima and sums; factors
    static constexpr int BARS = PARTS + 16 * N;             // scores, output, keys, values [2]
    static constexpr int THERE = BARS + 40;                 // chunks that exist: keys, values [2]
    static constexpr int START = THERE + 16;
    static constexpr int MORE = (START + 64 + 127) / 128 * 128;
    static constexpr int TMEM = GROUPS * (SIZE + MORE);     // tensor-memory address
    static constexpr int BYTES = TMEM + 16;
    // a group's tensor memory columns
    static constexpr uint32_t K_COL = 0, S_COL = D / 2, O_COL = S_COL + N, COLUMNS = O_COL + N;
    static constexpr int SLOT = N * (D + 3);                // floats of one partial result
    static_assert(SIZE % 1024 == 0 && BARS % 8 == 0 && START % 8 == 0 && sizeof(Start) <= 64, "layout");
    static_assert(BYTES <= 227 * 1024 && GROUPS * COLUMNS <= 512, "room");
};

// `bytes` of global memory to shared memory.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void load16(uint32_t at, uint32_t* r)
{
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ uint32_t load4(uint32_t at)
{
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(r) : "r"(at) : "memory");
    return r;
}

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
    unsigned char* more = smem_all + G::GROUPS * G::SIZE + group * G::MORE;
    const uint32_t sbase = smem_u32(smem), mbase = smem_u32(more);
    const uint32_t s_full = mbase + G::BARS, o_done = s_full + 8, k_full = s_full + 16, v_full = s_full + 24;
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem_all + G::TMEM);
    Start* start = reinterpret_cast<Start*>(more + G::START);
    // shares go to the SMs first, then to their groups
    const int share = group * gridDim.x + blockIdx.x;
    const int bar = 1 + group;

    if (row == 0) {
        for (int i = 0; i < 3 + G::VST; ++i)
            mbar_init(s_full + 8 * i, 1);
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
    // (all 512 columns are this CTA's, so they begin at 0)
    const uint32_t tm = group * G::COLUMNS, lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t k_at = tm + lanes + G::K_COL, s_at = tm + lanes + G::S_COL, o_at = tm + lanes + G::O_COL;
    bool ok = true;

    if (share < start->ctas) {
        uint64_t* words = reinterpret_cast<uint64_t*>(more + G::WORDS);
        int* pos = reinterpret_cast<int*>(more + G::POS);
        float* minus = reinterpret_cast<float*>(more + G::MINUS);
        float* parts = reinterpret_cast<float*>(more + G::PARTS);
        const int cs = kv4::chunk_shift(p.kv), page_mask = (1 << p.kv.page_shift) - 1;
        const int64_t page_bytes = kv4::page_bytes(p.kv);
        // where this key is held: its chunk of the block, its first row of codes and its first pair
        const int chunk = row >> cs, first = ((chunk * (D / 64) - chunk) << cs) + row;
        const uint32_t codes = mbase + first * 32, pairs = mbase + G::CODES + first * 4;
        // Its rows of V and of P, with the chunk 0 of their swizzles.  (Of V's codes the half
        // goes first that leaves the lanes' banks apart.)
        const int turn = (row >> 2) & 1;
        const uint32_t v_row = sbase + G::V + row * 128 + (((row & 7) ^ (turn << 2)) << 4);
        const uint32_t p_row = sbase + G::P + row * 32 + (turn << 4);
        // scores are c times the products; a scale of zero clears Q
        const float c = p.scale_log2 == 0.f ? 1.f : p.scale_log2;
        const float hidden = c < 0.f ? INFINITY : -INFINITY;
        auto wait = [&](uint32_t b, uint32_t parity) {
            if (ok)
                ok = mbar_wait(b, parity, p.wait_limit);
        };
        // The products, issued by a warp of the group: with the group as a constant every operand
        // is one, too (in registers of the threads' own they took some 130 instructions a
        // product, for which the other warps waited).
        const uint32_t sall = smem_u32(smem_all), mall = sall + G::GROUPS * G::SIZE;
        auto score = [&] {                                       // S^T = K Q^T
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < G::GROUPS; ++g)
                if (group == g) {
                    const uint64_t b = desc128(sall + g * G::SIZE + G::Q, 0);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        mma4_tk(g * G::COLUMNS + G::S_COL, g * G::COLUMNS + G::K_COL + h * 32, b + h * (G::QHALF >> 4),
                                idesc<DT>(N, false), h > 0);
                    commit(mall + g * G::MORE + G::BARS);
                }
        };
        auto value = [&](bool more) {                            // O^T (+)= V^T P^T
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < G::GROUPS; ++g)
                if (group == g) {
                    // (heads of 64 elements: the rows past them are what lies behind V, and not used)
                    const uint64_t a = desc128(sall + g * G::SIZE + G::V, G::HALF),
                                   b = desc32(sall + g * G::SIZE + G::P, G::PCHUNK);
#pragma unroll
                    for (int h = 0; h < 2; ++h)                  // 64 keys at a time
                        mma4_rr(g * G::COLUMNS + G::O_COL, a + h * 512, b + h * 128, idesc<DT>(N, true, true),
                                more || h > 0);
                    commit(mall + g * G::MORE + G::BARS + 8);
                }
        };
        Walk<S> w(p, *start, share);
        int n = 0;                                               // blocks so far
        int asked_k = 0, asked_v = 0;                            // copies so far (warp 3)
        while (w.next()) {
            const int rows = w.x.rows, nb = w.b_last - w.b_first, n0 = n;
            const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
            const uint8_t* base = kv4::chunk(p.kv, 0, w.head, 0);
            auto key0 = [&](int j) { return w.key0(w.b_first + j); };

            // ---- copies, by warp 3: lanes 2 i and 2 i + 1 have the codes and the pairs of chunk i ----
            auto page_of = [&](int j) {                          // the chunk's page in block j, -1: none
                const int key = key0(j) + ((lane >> 1) << cs);
                const bool in = j < nb && (lane >> 1) << cs < kKeys && wanted(p, w.x.lo, w.x.hi, key, 1 << cs);
                return in ? table[key >> p.kv.page_shift] : -1;
            };
            auto copy = [&](int which, int j, int page, int& asked) {
                if (j >= nb || !((unsigned)(n0 + j) < p.first_copies || share > 0))
                    return;                                      // (the test of the bounded waits)
                const bool go = page >= 0 && page < p.kv.pages;
                const unsigned there = __ballot_sync(0xffffffffu, go);
                const int st = which ? (n0 + j) % G::VST : 0;
                const uint32_t b = which ? v_full + st * 8 : k_full;
                const uint32_t size = lane & 1 ? 4 * (D / 64) << cs : 32 * (D / 64) << cs;
                if (lane == 0) {
                    reinterpret_cast<uint32_t*>(more + G::THERE)[which + st] = there;
                    mbar_expect_tx(b, (__popc(there) / 2) * (36 * (D / 64) << cs));
                }
                __syncwarp();
                if (go) {
                    const int s = (key0(j) + ((lane >> 1) << cs)) & page_mask;
                    const uint8_t* src = base + page * page_bytes + (s >> cs) * (kv4::slot_bytes(D) << cs) +
                                         (lane & 1 ? (D << cs) : 0) + which * size;
                    const uint32_t dst = mbase + (which ? G::VHELD + st * G::HELD : G::KHELD) +
                                         (lane & 1 ? G::CODES : 0) + (lane >> 1) * size;
                    bulk_copy(dst, src, size, b);
                }
                ++asked;
            };
            int page0 = -1, page1 = -1, page2 = -1;              // of the next blocks
            if (warp == 3) {
                page0 = page_of(0);
                page1 = page_of(1);
                copy(0, 0, page0, asked_k);
                copy(1, 0, page0, asked_v);
            }

            // ---- the queries, and what the rows see ----
            for (int i = row; i < rows * (D / 8); i += 128) {
                const int r = i / (D / 8), ch = i % (D / 8), qrow = w.x.row0 + r;
                const int t = token_of(p, qrow);
                const uint16_t* src = p.q + (int64_t)(w.q.q0 + t) * p.q_token +
                                      (int64_t)(w.head * p.group + qrow - t * p.group) * p.q_head + ch * 8;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (p.scale_log2 == 0.f) {
                } else if (p.q_wide) {
                    x = *reinterpret_cast<const uint4*>(src);
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
                minus[row] = kNone;
            }
            float2 x[N / 2];                                     // this key's share of the rows' sums
#pragma unroll
            for (int r = 0; r < N / 2; ++r)
                x[r] = make_float2(0.f, 0.f);
            // keys below `open_lo` or at `open_hi` and past are hidden from some row
            const int open_hi = p.tree ? min(w.q.keys, w.q.first)
                                       : min(w.q.keys, w.q.first + token_of(p, w.x.row0) + 1);
            const int open_lo =
                p.window > 0 ? w.q.first + token_of(p, w.x.row0 + rows - 1) - p.window + 1 : 0;
            if (warp == 3)
                page2 = page_of(2);

            // Whether block j's key (value) of this thread exists; slots past the context hold anything.
            auto there = [&](int which, int j) {
                const uint32_t mask = load4(mbase + G::THERE + 4 * which);
                return ((mask >> (2 * chunk)) & 1) && key0(j) + row < w.x.hi;
            };
            // Block j's key to tensor memory, and its scores asked for.
            auto key_in = [&](int j) {
                wait(k_full, (uint32_t)((n0 + j) & 1));
                const bool is = there(0, j);
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    const uint32_t sb = is ? load4(pairs + G::KHELD + (part * 4 << cs)) : 0u;
                    const uint32_t sc = kv4::both_scales(sb), bi = kv4::both_biases(sb);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t held[4], e[16];
                        load16(codes + G::KHELD + (part * 32 << cs) + h * 16, held);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            kv4::expand<DT>(held[i], sc, bi, reinterpret_cast<uint32_t(&)[4]>(e[4 * i]));
                        tmem_st16(k_at + part * 32 + h * 16, e);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(bar, 128);                        // K is read and in
                if (warp == 0)
                    score();
            };
            // Its value to shared memory, when the last block's has been used.
            auto value_in = [&](int j) {
                if (n0 + j > 0)
                    wait(o_done, (uint32_t)((n0 + j - 1) & 1));
                const int st = (n0 + j) % G::VST;
                wait(v_full + st * 8, (uint32_t)(((n0 + j) / G::VST) & 1));
                const bool is = there(1 + st, j);
                const uint32_t at = G::VHELD + st * G::HELD;
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    const uint32_t sb = is ? load4(pairs + at + (part * 4 << cs)) : 0u;
                    const uint32_t sc = kv4::both_scales(sb), bi = kv4::both_biases(sb);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t held[4];
                        load16((codes + at + (part * 32 << cs)) ^ ((turn ^ h) << 4), held);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t e[4];
                            kv4::expand<DT>(held[i], sc, bi, e);
                            store16((v_row ^ ((4 * h + i) << 4)) + part * G::HALF, e);
                        }
                    }
                }
            };
            float t[16];
            // scores of 16 rows
            auto scores = [&](int ch, int k0) {
                tmem_ld16(s_at + ch * 16, t);
                tmem_wait_ld();
                if (k0 + kKeys > open_hi || k0 < open_lo) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (!sees(p, w.q, pos[ch * 16 + i], words[ch * 16 + i], k0 + row))
                            t[i] = hidden;
                }
            };
            // exponents of two of the chunk's rows, and the largest of those of 8 rows
            auto exponents = [&](int ch, int at) {
                return fma2(make_float2(t[at], t[at + 1]), make_float2(c, c),
                            *reinterpret_cast<const float2*>(minus + ch * 16 + at));
            };
            auto larger = [&](float top, float2 e, int r) {
                if (r < rows)
                    top = fmaxf(top, e.x);
                if (r + 1 < rows)
                    top = fmaxf(top, e.y);
                return top;
            };
            // Probabilities of 8 rows from h * 8 on of the chunk, kept and as a part of the key's row
            // of P; the largest of their exponents.
            float2 weight[CH == 1 ? 8 : 4];
            auto weigh = [&](int ch, int h) {
                float top = -INFINITY;
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = exponents(ch, h * 8 + 2 * i);
                    top = larger(top, e, ch * 16 + h * 8 + 2 * i);
                    float2& y = weight[(CH == 1 ? h * 4 : 0) + i];
                    y = make_float2(ex2(e.x), ex2(e.y));
                    r[i] = pack2<DT>(y.x, y.y);
                }
                store16((p_row ^ (h << 4)) + ch * G::PCHUNK, r);
                return top;
            };
            auto add = [&](int ch, int h) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[ch * 8 + h * 4 + i] = add2(x[ch * 8 + h * 4 + i], weight[(CH == 1 ? h * 4 : 0) + i]);
            };
            // Moves the references that the block's maxima pass by more than 8, and the sums with
            // them.  (Of more than a chunk the scores are in tensor memory still.)
            auto move = [&](int j) {
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
                    if (ch * 16 < rows) {
                        if (CH > 1)
                            scores(ch, key0(j));
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float most = warp_max(t[i] * c);
                            if (lane == 0)
                                parts[warp * N + ch * 16 + i] = most;
                        }
                    }
                named_bar_sync(bar, 128);
                if (row < rows) {
                    float* q = parts + row;
                    const float most = fmaxf(fmaxf(q[0], q[N]), fmaxf(q[2 * N], q[3 * N]));
                    float f = 1.f;
                    if (most + minus[row] > 8.f) {
                        f = ex2(-minus[row] - most);
                        minus[row] = -most;
                    }
                    q[0] = f;                                    // the factor of the row's sums
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
                            const float f = ch * 16 + i < rows ? parts[ch * 16 + i] : 1.f;
                            (i & 1 ? x[ch * 8 + i / 2].y : x[ch * 8 + i / 2].x) *= f;
                            r[i] = __float_as_uint(o[i] * f);
                        }
                        if (j > 0)
                            tmem_st16(o_at + ch * 16, r);
                    }
                tmem_wait_st();
            };

            if (CH == 1) {
                // A block's scores are computed while the block before it is weighed: they stay
                // in registers, and the next key takes their place.
#pragma unroll 1
                for (int j = -1; j < nb; ++j) {
                    if (j >= 0) {
                        wait(s_full, (uint32_t)((n0 + j) & 1));
                        tc_fence_after();
                        scores(0, key0(j));
                    }
                    if (j + 1 < nb) {
                        key_in(j + 1);
                        if (warp == 3) {
                            copy(0, j + 2, page1, asked_k);
                            if (j >= 0)                          // its stage's last use is over
                                copy(1, j + 1, page0, asked_v);
                            page0 = page1;
                            page1 = page2;
                            page2 = page_of(j + 4);
                        }
                    }
                    if (j < 0)
                        continue;
                    value_in(j);
                    float top = weigh(0, 0);
                    if (rows > 8)
                        top = fmaxf(top, weigh(0, 1));
                    fence_proxy_async_smem();
                    tc_fence_before();
                    if (any_of_group(bar, top > 8.f)) {
                        move(j);
                        weigh(0, 0);
                        if (rows > 8)
                            weigh(0, 1);
                        fence_proxy_async_smem();
                        tc_fence_before();
                        named_bar_sync(bar, 128);
                    }
                    add(0, 0);
                    if (rows > 8)
                        add(0, 1);
                    if (warp == 1)
                        value(j > 0);
                }
            } else {
                // of more rows the scores stay in tensor memory: their exponents are looked at, and
                // then weighed
#pragma unroll 1
                for (int j = 0; j < nb; ++j) {
                    key_in(j);
                    if (warp == 3)
                        copy(0, j + 1, page1, asked_k);
                    value_in(j);
                    wait(s_full, (uint32_t)((n0 + j) & 1));
                    tc_fence_after();
                    float top = -INFINITY;
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch)
                        if (ch * 16 < rows) {
                            scores(ch, key0(j));
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                top = larger(top, exponents(ch, 2 * i), ch * 16 + 2 * i);
                        }
                    const bool moved = any_of_group(bar, top > 8.f);
                    if (warp == 3) {                             // V is read
                        copy(1, j + 1, page1, asked_v);
                        page1 = page2;
                        page2 = page_of(j + 3);
                    }
                    if (moved)
                        move(j);
#pragma unroll
                    for (int ch = 0; ch < CH; ++ch)
                        if (ch * 16 < rows) {
                            scores(ch, key0(j));
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (ch * 16 + h * 8 < rows) {
                                    weigh(ch, h);
                                    add(ch, h);
                                }
                        }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    named_bar_sync(bar, 128);
                    if (warp == 1)
                        value(j > 0);
                }
            }
            n += nb;

            // ---- the item's result: a thread has an element of every row ----
#pragma unroll
            for (int r = 0; r < N; ++r)
                if (r < rows) {
                    float s = r & 1 ? x[r / 2].y : x[r / 2].x;
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
                    slot[N * D + row] = -minus[row];
                    slot[N * (D + 1) + row] = slot[N * (D + 2) + row] = s;
                } else if (p.lse) {
                    const int qrow = w.x.row0 + row, tok = token_of(p, qrow);
                    p.lse[(int64_t)(w.q.q0 + tok) * p.heads + w.head * p.group + qrow - tok * p.group] =
                        lse_of(-minus[row], s);
                }
            }
            if (!whole && row == 0 && c0 == share)
                static_cast<JoinItem*>(p.items)[c0] = {w.q.q0, w.x.row0, rows, w.head, c1 - c0 + 1};
            tc_fence_before();
            named_bar_sync(bar, 128);                            // what the rows need has been read
        }
        // the last products and copies end before tensor and shared memory go away, also after a
        // wait that ran out
        bool end = true;
        if (n > 0)
            end = mbar_wait(s_full, (uint32_t)((n - 1) & 1), p.wait_limit) &&
                  mbar_wait(o_done, (uint32_t)((n - 1) & 1), p.wait_limit);
        if (asked_k > 0)
            end = mbar_wait(k_full, (uint32_t)((asked_k - 1) & 1), p.wait_limit) && end;
        for (int i = asked_v - 1; i >= 0 && i >= asked_v - G::VST; --i)
            end = mbar_wait(v_full + i % G::VST * 8, (uint32_t)((i / G::VST) & 1), p.wait_limit) && end;
        ok = ok && end;
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
    return launch<DT, D, 16>(p, sms, st);
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

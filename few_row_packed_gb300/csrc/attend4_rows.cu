// attend4_rows.cu -- attention of few new tokens over a paged cache of 4 bits (plain
// decoding, verify calls, trees of drafted tokens).
//
// The sums of attend_rows.cu.  A quarter of the bytes leaves a quarter of the time for
// everything else, so the products are turned around: keys are the 128 rows of the
// tensor core's tile and the queries, a few, its columns,
//     S^T = K Q^T (128 keys x N rows),   O^T += V^T P^T (D x N rows).
// An MMA's time then goes by its operands' bytes, not by padded rows, and
//   * two threads have a key, half of its elements and half of the rows each.  They expand
//     its codes and write it to tensor memory, where the first product takes it from; they
//     get its scores from there, mask them, take the exponentials, and add them up for
//     themselves, one sum a row, joined with the other keys' at the item's end;
//   * they write its values and probabilities to shared memory as a row each, which are
//     the second product's operands as they are: rows along the contracted dimension.
// A group of eight such warps does this block by block for a share of its own, with a
// warp beside it that copies the codes a block ahead (bulk copies: a chunk's keys, values
// and scales are stretches of memory) and issues the products.  The groups of a CTA
// have nothing to do with one another but the SM, whose schedulers take one's arithmetic while
// another waits.  Shares, items and references are those of attend_common.cuh (a reference
// moves when a score passes it by more than 8); the parts of divided items are added by a
// launch of their own (attend_join.cu).
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

constexpr int kKeys = 128;                       // keys per block
constexpr int kTeam = 256;                       // threads of a group, without its warp for copies
constexpr int kGroups = 3;
// Units of a block and of an item beside its blocks; the least share of a group.
constexpr int kBlockUnits = 4, kExtra = 6, kMinUnits = 4;
// A reference that every score passes, negated: nothing has been seen yet.
constexpr float kNone = 1e30f;
constexpr int kItems = 4;                        // items known at a time: of three blocks, and one more

// What a group needs to know of an item.
struct alignas(16) Item {
    int q0, first, keys;   // of its request
    int row0, rows, head, hi, r;
    int key0, nb;          // its first key and its blocks in this share; 0 blocks: no more items
    int skip, jump;        // keys left out before block `jump` (behind the sinks)
    int c0, c1;            // shares that hold a part of it
    int unused[2];
    __device__ int key_of(int j) const { return key0 + j * kKeys + (j >= jump ? skip : 0); }
};
static_assert(sizeof(Item) == 64, "ring entry");

// N: rows of an item, 16 or 48.
template <int D, int N>
struct Geo4 {
    static constexpr int VST = N == 16 ? 2 : 1;             // stages of values as they are held
    static constexpr int THREADS = kGroups * (kTeam + 32);
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
    static constexpr int ITEMS = VHELD + VST * HELD;
    static constexpr int START = ITEMS;                     // where the share begins, before its first item
    static constexpr int POS = ITEMS + kItems * 64;         // int [N]: the rows' positions
    static constexpr int MINUS = POS + 4 * N;               // float [N]: their references, negated
    static constexpr int PARTS = MINUS + 4 * N;             // [4][N]: warps' maxima and sums; factors
    static constexpr int BARS = PARTS + 16 * N;
    static constexpr int NBARS = 7 + kItems;
    static constexpr int THERE = BARS + 8 * NBARS;          // chunks that exist: keys, values [2]
    static constexpr int MORE = (THERE + 12 + 31) / 32 * 32;
    static constexpr int TMEM = kGroups * (SIZE + MORE);    // tensor-memory address
    static constexpr int BYTES = TMEM + 16;
    // a group's tensor memory columns
    static constexpr uint32_t K_COL = 0, S_COL = D / 2, O_COL = S_COL + N, COLUMNS = O_COL + N;
    static constexpr int SLOT = N * (D + 3);                // floats of one partial result
    static_assert(SIZE % 1024 == 0 && ITEMS % 16 == 0 && BARS % 8 == 0 && sizeof(Start) <= kItems * 64, "layout");
    static_assert(BYTES <= 227 * 1024 && kGroups * COLUMNS <= 512, "room");
};

// mbar_wait after a try that failed, for waits that are long as a rule: out of line of the
// code around it, and the warp sleeps up to 0.1 ms at a time.
__device__ __noinline__ bool mbar_sleep(uint32_t bar, uint32_t parity, unsigned limit)
{
    const long long t0 = clock64();
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(100000u)
            : "memory");
        if (ok)
            return true;
        if (clock64() - t0 > (long long)limit)
            return false;
    }
}

// `bytes` of global memory to shared memory.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void load16(uint32_t at, uint32_t (&r)[4])
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

__device__ __forceinline__ void store8(uint32_t at, uint32_t a, uint32_t b)
{
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};\n" ::"r"(at), "r"(a), "r"(b) : "memory");
}

// Whether any of the group's threads says so; all of them meet here.
__device__ __forceinline__ bool any_of_group(int bar, bool mine)
{
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %2, 0;\n bar.red.or.pred q, %1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
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
    constexpr bool kAhead = N == 16;             // scores stay in registers, the next key's are asked for early
    constexpr int NC = N / 8;                    // 8 rows at a time, 4 of them a thread's
    extern __shared__ __align__(1024) unsigned char smem_all[];
    const int tid = threadIdx.x, lane = tid & 31;
    const bool helper = tid >= kGroups * kTeam;  // the warp beside a group
    const int group = helper ? (tid - kGroups * kTeam) >> 5 : tid / kTeam;
    const int row = tid & 127, half = (tid >> 7) & 1, warp = (tid >> 5) & 3;   // key; part of it; lanes of tensor memory
    unsigned char* smem = smem_all + group * G::SIZE;
    unsigned char* more = smem_all + kGroups * G::SIZE + group * G::MORE;
    const uint32_t sbase = smem_u32(smem), mbase = smem_u32(more);
    auto bar_at = [&](int i) { return mbase + G::BARS + 8 * i; };
    const uint32_t s_full = bar_at(0), o_done = bar_at(1);   // products are complete
    const uint32_t k_in = bar_at(2), p_in = bar_at(3);       // their operands are there
    const uint32_t k_full = bar_at(4), v_full = bar_at(5);   // copies have arrived (v_full: two)
    auto item_full = [&](int i) { return bar_at(7 + i % kItems); };
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem_all + G::TMEM);
    Item* items = reinterpret_cast<Item*>(more + G::ITEMS);
    const int share = group * gridDim.x + blockIdx.x;        // the SMs first, then their groups

    if (helper && lane == 0) {
        for (int i = 0; i < G::NBARS; ++i)
            mbar_init(bar_at(i), i == 2 ? 8 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid < 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    after_previous();
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) {
        if (!mbar_try(b, parity) && ok)
            ok = mbar_sleep(b, parity, p.wait_limit);
    };
    const int cs = kv4::chunk_shift(p.kv);

    if (helper) {
        // ---- copies and products ----
        if (lane == 0)
            static_cast<JoinItem*>(p.items)[share].rows = 0;
        Start* start = reinterpret_cast<Start*>(more + G::START);
        find_start<S>(p, lane, gridDim.x * kGroups, kMinUnits, share, start);
        __syncwarp();
        const Start begin = *start;
        __syncwarp();
        int published = 0;
        auto publish = [&](const Item& x) {                  // by lane 0
            items[published % kItems] = x;
            mbar_arrive(item_full(published));               // releases the stores
        };
        if (share >= begin.ctas) {                           // fewer units than groups
            if (lane == 0) {
                Item none = {};
                publish(none);
            }
        } else {
            const int page_mask = (1 << p.kv.page_shift) - 1;
            const int64_t page_bytes = kv4::page_bytes(p.kv);
            // lanes 2 i and 2 i + 1 have the codes and the pairs of chunk i
            const int chunk0 = (lane >> 1) << cs;
            const uint32_t size = lane & 1 ? 4 * (D / 64) << cs : 32 * (D / 64) << cs;
            Walk<S> w(p, begin, share);
            // A block of the share: where this lane's chunk of it lies, if it exists.
            struct Block {
                int page, offset, head;
                bool any, first, last, full;                 // full: every key of it exists
            };
            int j = 0, nb = 0;                               // of the item that `ahead` is of
            auto next_block = [&]() -> Block {
                Block x = {-1, 0, 0, true, false, false, false};
                if (++j >= nb) {
                    x.any = w.next();
                    j = 0;
                    nb = x.any ? w.b_last - w.b_first : 0;
                    x.first = true;
                    if (lane == 0) {
                        const bool split = w.b_first < w.x.near;     // sinks, then a window
                        const bool whole = w.whole();
                        Item it = {w.q.q0, w.q.first, w.q.keys, w.x.row0, w.x.rows, w.head, w.x.hi, w.r,
                                   w.key0(w.b_first), nb, split ? w.x.gap * kKeys : 0, w.x.near - w.b_first,
                                   whole ? 0 : w.first_cta(), whole ? 0 : w.last_cta(), {0, 0}};
                        publish(it);
                    }
                    ++published;
                }
                if (x.any) {
                    const int key = w.key0(w.b_first + j) + chunk0;
                    if (chunk0 < kKeys && wanted(p, w.x.lo, w.x.hi, key, 1 << cs))
                        x.page = p.batch.block_table[(int64_t)w.r * p.batch.table_stride + (key >> p.kv.page_shift)];
                    x.offset = ((key & page_mask) >> cs) * (kv4::slot_bytes(D) << cs) + (lane & 1 ? D << cs : 0);
                    x.head = w.head;
                    x.last = j + 1 == nb;
                    x.full = w.key0(w.b_first + j) + kKeys <= w.x.hi;
                }
                return x;
            };
            // Copies its keys (0) or values (1).  (The test of the bounded waits leaves some out.)
            int asked_k = 0, asked_v = 0;
            auto copy = [&](int which, const Block& x, int& asked) {
                if (!x.any || !((unsigned)asked < p.first_copies || share > 0))
                    return;
                const bool go = x.page >= 0 && x.page < p.kv.pages;
                const unsigned there = __ballot_sync(0xffffffffu, go);
                const int st = which ? asked % G::VST : 0;
                const uint32_t b = which ? v_full + st * 8 : k_full;
                if (lane == 0) {
                    const int chunks = __popc(there) / 2;
                    reinterpret_cast<uint32_t*>(more + G::THERE)[which + st] =
                        x.full && chunks == kKeys >> cs ? ~0u : there & 0x55555555u;
                    mbar_expect_tx(b, chunks * (36 * (D / 64) << cs));
                }
                __syncwarp();
                if (go)
                    bulk_copy(mbase + (which ? G::VHELD + st * G::HELD : G::KHELD) + (lane & 1 ? G::CODES : 0) +
                                  (lane >> 1) * size,
                              kv4::chunk(p.kv, 0, x.head, 0) + x.page * page_bytes + x.offset + which * size, size, b);
                ++asked;
            };
            // The products: with the group as a constant every operand is one, too (in registers
            // of the threads' own they took some 130 instructions a product).
            const uint32_t sall = smem_u32(smem_all), mall = sall + kGroups * G::SIZE;
            auto score = [&](int n) {                        // S^T = K Q^T
                wait(k_in, (uint32_t)(n & 1));
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    if (group == g) {
                        const uint64_t b = desc128(sall + g * G::SIZE + G::Q, 0);
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            mma4_tk(g * G::COLUMNS + G::S_COL, g * G::COLUMNS + G::K_COL + h * 32,
                                    b + h * (G::QHALF >> 4), idesc<DT>(N, false), h > 0);
                        commit(mall + g * G::MORE + G::BARS);
                    }
            };
            auto value = [&](int n, bool add) {              // O^T (+)= V^T P^T
                wait(p_in, (uint32_t)(n & 1));
                __syncwarp();
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                    if (group == g) {
                        // (heads of 64 elements: the rows past them are what lies behind V, and not used)
                        const uint64_t a = desc128(sall + g * G::SIZE + G::V, G::HALF),
                                       b = desc32(sall + g * G::SIZE + G::P, G::PCHUNK);
#pragma unroll
                        for (int h = 0; h < 2; ++h)          // 64 keys at a time
                            mma4_rr(g * G::COLUMNS + G::O_COL, a + h * 512, b + h * 128, idesc<DT>(N, true, true),
                                    add || h > 0);
                        commit(mall + g * G::MORE + G::BARS + 8);
                    }
            };
            Block now = next_block(), ahead;                 // blocks n and n + 1
            copy(0, now, asked_k);
            copy(1, now, asked_v);
            ahead = next_block();
            bool before = false;                             // block n - 1 was its item's first
            int n = 0, scored = 0, valued = 0;
            // (After a wait that ran out nothing more is published: the group's warps may be
            // anywhere in the items that it knows.)
            auto fine = [&] { return ok = __all_sync(0xffffffffu, ok); };
            for (; now.any; ++n) {
                score(n);
                ++scored;
                if (!fine())
                    break;
                copy(0, ahead, asked_k);                     // the keys have been read
                const Block after = ahead.any ? next_block() : ahead;
                if (kAhead && !now.first)
                    value(n - 1, !before), ++valued;
                if (kAhead)
                    copy(1, ahead, asked_v);                 // its stage's last use is over
                if (!kAhead || now.last)
                    value(n, !now.first), ++valued;
                if (!kAhead)
                    copy(1, ahead, asked_v);
                if (!fine())
                    break;
                before = now.first;
                now = ahead;
                ahead = after;
            }
            // the last products and copies end before tensor and shared memory go away, also
            // after a wait that ran out
            __syncwarp();
            bool end = true;
            if (scored > 0)
                end = mbar_wait(s_full, (uint32_t)((scored - 1) & 1), p.wait_limit);
            if (valued > 0)
                end = mbar_wait(o_done, (uint32_t)((valued - 1) & 1), p.wait_limit) && end;
            if (asked_k > 0)
                end = mbar_wait(k_full, (uint32_t)((asked_k - 1) & 1), p.wait_limit) && end;
            for (int i = asked_v - 1; i >= 0 && i >= asked_v - G::VST; --i)
                end = mbar_wait(v_full + i % G::VST * 8, (uint32_t)((i / G::VST) & 1), p.wait_limit) && end;
            ok = ok && end;
        }
    } else {
        // ---- the keys ----
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        // (all 512 columns are this CTA's, so they begin at 0)
        const uint32_t tm = group * G::COLUMNS + lanes;
        const uint32_t k_at = tm + G::K_COL + half * (D / 4), s_at = tm + G::S_COL + half * 4,
                       o_at = tm + G::O_COL + half * 4;
        const int bar = 1 + group;
        int* pos = reinterpret_cast<int*>(more + G::POS);
        float* minus = reinterpret_cast<float*>(more + G::MINUS);
        float* parts = reinterpret_cast<float*>(more + G::PARTS);
        // where this key is held: its chunk of the block, this half's first row of codes and pair
        constexpr int W = D / 64;                            // vectors of 16 bytes of codes a thread has
        const int chunk = row >> cs, first = ((chunk * (D / 64) - chunk) << cs) + row + (D == 128 ? half << cs : 0);
        const uint32_t codes = mbase + first * 32 + (D == 64 ? half * 16 : 0), pairs = mbase + G::CODES + first * 4;
        // Its rows of V and of P, with the chunk 0 of their swizzles.  (Of V's two vectors of codes
        // the one goes first that leaves the lanes' banks apart.)
        const int turn = (row >> 2) & 1, swap = D == 128 ? turn : 0;
        const uint32_t v_row = sbase + G::V + (D == 128 ? half * G::HALF : 0) + row * 128 +
                               (((row & 7) ^ (D == 128 ? swap << 2 : half << 2)) << 4);
        const uint32_t p_row = sbase + G::P + row * 32 + (turn << 4) + half * 8;
        // scores are c times the products; a scale of zero clears Q
        const float c = p.scale_log2 == 0.f ? 1.f : p.scale_log2;
        const float hidden = c < 0.f ? INFINITY : -INFINITY;
        const kv4::Constants constants = kv4::constants<DT>();
        int n0 = 0;                                          // blocks before the item
        for (int it = 0;; ++it) {
            // one warp waits for the item, and all of them hear whether it came
            bool stop = false;
            if (half == 0 && warp == 0) {
                wait(item_full(it), (uint32_t)((it / kItems) & 1));
                stop = !ok || items[it % kItems].nb == 0;
            }
            if (any_of_group(bar, stop))
                break;
            const Item& w = items[it % kItems];
            const int rows = w.rows, nb = w.nb, hi = w.hi;
            // the queries (zeros for the rows that fill up 8), and what the rows see
            for (int i = tid % kTeam; i < (rows + 7) / 8 * 8 * (D / 8); i += kTeam) {
                const int r = i / (D / 8), ch = i % (D / 8), qrow = w.row0 + r;
                const int t = token_of(p, qrow);
                const uint16_t* src = p.q + (int64_t)(w.q0 + t) * p.q_token +
                                      (int64_t)(w.head * p.group + qrow - t * p.group) * p.q_head + ch * 8;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (p.scale_log2 == 0.f || r >= rows) {
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
            if (tid % kTeam < N) {
                const int r = tid % kTeam, i = token_of(p, w.row0 + r);
                pos[r] = r < rows ? w.first + i : INT_MIN / 2;
                minus[r] = r < rows ? kNone : 0.f;
            }
            named_bar_sync(bar, kTeam);
            float2 x[2 * NC];                                // this key's share of the rows' sums
#pragma unroll
            for (int i = 0; i < 2 * NC; ++i)
                x[i] = make_float2(0.f, 0.f);
            // keys below `open_lo` or at `open_hi` and past are hidden from some row
            const int open_hi = p.tree ? min(w.keys, w.first) : min(w.keys, w.first + token_of(p, w.row0) + 1);
            const int open_lo = p.window > 0 ? w.first + token_of(p, w.row0 + rows - 1) - p.window + 1 : 0;

            // A thread's (scale, bias) of a plane, zeros where its key does not exist: slots past the
            // context hold anything.  (All ones: every key of the block exists.)
            auto pair_of = [&](int which, uint32_t at, int j) {
                const uint32_t mask = load4(mbase + G::THERE + 4 * which);
                uint32_t sb = load4(pairs + at);
                if (mask != ~0u)
                    sb = ((mask >> (2 * chunk)) & 1) && w.key_of(j) + row < hi ? sb : 0u;
                return sb;
            };
            // Block j's key to tensor memory, and its scores asked for.
            auto key_in = [&](int j) {
                wait(k_full, (uint32_t)(n0 + j) & 1);
                const uint32_t sb = pair_of(0, G::KHELD, j);
                const uint32_t sc = kv4::both_scales(sb), bi = kv4::both_biases(sb);
#pragma unroll
                for (int h = 0; h < W; ++h) {
                    uint32_t held[4], e[16];
                    load16(codes + G::KHELD + h * 16, held);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        kv4::expand<DT>(held[i], sc, bi, constants, reinterpret_cast<uint32_t(&)[4]>(e[4 * i]));
                    tmem_st16(k_at + h * 16, e);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(k_in);
            };
            // Its value to shared memory, when the last block's has been used.
            auto value_in = [&](int j) {
                if (n0 + j > 0)
                    wait(o_done, (uint32_t)((n0 + j - 1) & 1));
                const int st = (n0 + j) % G::VST;
                wait(v_full + st * 8, (uint32_t)(((n0 + j) / G::VST) & 1));
                const uint32_t at = G::VHELD + st * G::HELD, sb = pair_of(1 + st, at, j);
                const uint32_t sc = kv4::both_scales(sb), bi = kv4::both_biases(sb);
#pragma unroll
                for (int h = 0; h < W; ++h) {
                    uint32_t held[4];
                    load16((codes + at) ^ ((swap ^ h) << 4), held);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t e[4];
                        kv4::expand<DT>(held[i], sc, bi, constants, e);
                        store16(v_row ^ ((4 * h + i) << 4), e);
                    }
                }
            };
            // scores of this thread's 4 of 8 rows
            auto scores = [&](int ch, float (&t)[4], int k0) {
                tmem_ld4(s_at + ch * 8, t);
                tmem_wait_ld();
                if (k0 > open_hi - kKeys || k0 < open_lo) {
                    Request q;
                    q.first = w.first, q.keys = w.keys;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = ch * 8 + half * 4 + i;
                        const uint64_t word = p.tree && r < rows ? p.tree[w.q0 + pos[r] - w.first] : 0;
                        if (!sees(p, q, pos[r], word, k0 + row))
                            t[i] = hidden;
                    }
                }
            };
            // their exponents, two at a time
            auto exponents = [&](int ch, int i, const float (&t)[4]) {
                return fma2(make_float2(t[2 * i], t[2 * i + 1]), make_float2(c, c),
                            *reinterpret_cast<const float2*>(minus + ch * 8 + half * 4 + 2 * i));
            };
            // Their probabilities, kept in y and as a part of the key's row of P; the largest exponent.
            auto weigh = [&](int ch, const float (&t)[4], float2 (&y)[2]) {
                const float2 a = exponents(ch, 0, t), b = exponents(ch, 1, t);
                y[0] = make_float2(ex2(a.x), ex2(a.y));
                y[1] = make_float2(ex2(b.x), ex2(b.y));
                store8((p_row ^ ((ch & 1) << 4)) + (ch >> 1) * G::PCHUNK, pack2<DT>(y[0].x, y[0].y),
                       pack2<DT>(y[1].x, y[1].y));
                return fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
            };
            auto add = [&](int ch, const float2 (&y)[2]) {
                x[2 * ch] = add2(x[2 * ch], y[0]);
                x[2 * ch + 1] = add2(x[2 * ch + 1], y[1]);
            };
            // Moves the references that the block's maxima pass by more than 8, and the sums with them.
            auto most_of = [&](int ch, const float (&t)[4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float most = warp_max(t[i] * c);
                    if (lane == 0)
                        parts[warp * N + ch * 8 + half * 4 + i] = most;
                }
            };
            auto move = [&](int j) {
                named_bar_sync(bar, kTeam);
                if (tid % kTeam < rows) {
                    float *q = parts + tid % kTeam, *m = minus + tid % kTeam;
                    const float most = fmaxf(fmaxf(q[0], q[N]), fmaxf(q[2 * N], q[3 * N]));
                    float f = 1.f;
                    if (most + *m > 8.f) {
                        f = ex2(-*m - most);
                        *m = -most;
                    }
                    q[0] = f;                                // the factor of the row's sums
                }
                named_bar_sync(bar, kTeam);
#pragma unroll
                for (int ch = 0; ch < NC; ++ch)
                    if (ch * 8 < rows) {
                        float o[4], f[4];
                        if (j > 0) {
                            tmem_ld4(o_at + ch * 8, o);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = ch * 8 + half * 4 + i;
                            f[i] = r < rows ? parts[r] : 1.f;
                            o[i] *= f[i];
                        }
                        x[2 * ch].x *= f[0], x[2 * ch].y *= f[1];
                        x[2 * ch + 1].x *= f[2], x[2 * ch + 1].y *= f[3];
                        if (j > 0)
                            tmem_st4(o_at + ch * 8, o);
                    }
                tmem_wait_st();
            };
            auto done = [&] {                                // P and V are in: by one thread, after the others
                if (tid % kTeam == 0)
                    mbar_arrive(p_in);
            };

            if (kAhead) {
                // A block's scores are computed while the block before it is weighed: they stay
                // in registers, and the next key takes their place.
                key_in(0);
#pragma unroll 1
                for (int j = 0; j < nb; ++j) {
                    float t[NC][4];
                    float2 y[NC][2];
                    wait(s_full, (uint32_t)((n0 + j) & 1));
                    tc_fence_after();
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch)
                        if (ch * 8 < rows)
                            scores(ch, t[ch], w.key_of(j));
                    if (j + 1 < nb)
                        key_in(j + 1);
                    value_in(j);
                    float top = -INFINITY;
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch)
                        if (ch * 8 < rows)
                            top = fmaxf(top, weigh(ch, t[ch], y[ch]));
                    fence_proxy_async_smem();
                    tc_fence_before();
                    if (any_of_group(bar, top > 8.f)) {
#pragma unroll
                        for (int ch = 0; ch < NC; ++ch)
                            if (ch * 8 < rows)
                                most_of(ch, t[ch]);
                        move(j);
#pragma unroll
                        for (int ch = 0; ch < NC; ++ch)
                            if (ch * 8 < rows)
                                weigh(ch, t[ch], y[ch]);
                        fence_proxy_async_smem();
                        tc_fence_before();
                        named_bar_sync(bar, kTeam);
                    }
                    done();
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch)
                        if (ch * 8 < rows)
                            add(ch, y[ch]);
                }
            } else {
                // of more rows the scores stay in tensor memory: their exponents are looked at, and
                // then weighed
#pragma unroll 1
                for (int j = 0; j < nb; ++j) {
                    const int k0 = w.key_of(j);
                    float t[4];
                    key_in(j);
                    value_in(j);
                    wait(s_full, (uint32_t)((n0 + j) & 1));
                    tc_fence_after();
                    float top = -INFINITY;
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch)
                        if (ch * 8 < rows) {
                            scores(ch, t, k0);
                            const float2 a = exponents(ch, 0, t), b = exponents(ch, 1, t);
                            top = fmaxf(top, fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)));
                        }
                    if (any_of_group(bar, top > 8.f)) {
#pragma unroll
                        for (int ch = 0; ch < NC; ++ch)
                            if (ch * 8 < rows) {
                                scores(ch, t, k0);
                                most_of(ch, t);
                            }
                        move(j);
                    }
#pragma unroll
                    for (int ch = 0; ch < NC; ++ch)
                        if (ch * 8 < rows) {
                            float2 y[2];
                            scores(ch, t, k0);
                            weigh(ch, t, y);
                            add(ch, y);
                        }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    named_bar_sync(bar, kTeam);
                    done();
                }
            }
            n0 += nb;

            // ---- the item's result: a thread has an element of its rows ----
#pragma unroll
            for (int ch = 0; ch < NC; ++ch)
                if (ch * 8 < rows) {
                    float s[4] = {x[2 * ch].x, x[2 * ch].y, x[2 * ch + 1].x, x[2 * ch + 1].y};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1)
                            s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
                        if (lane == 0)
                            parts[warp * N + ch * 8 + half * 4 + i] = s[i];
                    }
                }
            named_bar_sync(bar, kTeam);
            wait(o_done, (uint32_t)((n0 - 1) & 1));
            tc_fence_after();
            const bool whole = w.c0 == w.c1;
            float* slot = p.partial + (size_t)(2 * share + (w.c0 == share)) * G::SLOT;
            auto sum_of = [&](int r) { return (parts[r] + parts[N + r]) + (parts[2 * N + r] + parts[3 * N + r]); };
#pragma unroll
            for (int ch = 0; ch < NC; ++ch)
                if (ch * 8 < rows) {
                    float o[4];
                    tmem_ld4(o_at + ch * 8, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = ch * 8 + half * 4 + i;
                        if (r < rows && row < D) {
                            if (whole) {
                                const int qrow = w.row0 + r, tok = token_of(p, qrow);
                                const float s = sum_of(r);
                                const uint32_t y = s > 0.f ? pack2<DT>(o[i] / s, 0.f) : 0u;
                                p.out[(int64_t)(w.q0 + tok) * p.out_token +
                                      (int64_t)(w.head * p.group + qrow - tok * p.group) * p.out_head + row] =
                                    (uint16_t)y;
                            } else {
                                slot[r * D + row] = o[i];
                            }
                        }
                    }
                }
            if (tid % kTeam < rows) {
                const int r = tid % kTeam;
                const float s = sum_of(r);
                if (!whole) {
                    slot[N * D + r] = -minus[r];
                    slot[N * (D + 1) + r] = slot[N * (D + 2) + r] = s;
                } else if (p.lse) {
                    const int qrow = w.row0 + r, tok = token_of(p, qrow);
                    p.lse[(int64_t)(w.q0 + tok) * p.heads + w.head * p.group + qrow - tok * p.group] =
                        lse_of(-minus[r], s);
                }
            }
            if (!whole && tid % kTeam == 0 && w.c0 == share)
                static_cast<JoinItem*>(p.items)[w.c0] = {w.q0, w.row0, rows, w.head, w.c1 - w.c0 + 1};
            tc_fence_before();
            named_bar_sync(bar, kTeam);                      // what the rows need has been read
        }
    }
    if (!ok)
        atomicOr(p.status, 1u);
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
    const int ctas = std::min(sms, kAttendMaxCtas / kGroups);
    e = launch_after(kernel, dim3((unsigned)ctas), G::THREADS, G::BYTES, st, p);
    return e == cudaSuccess ? launch_attend_join(p, (lbv_dtype)DT, N, ctas * kGroups, st) : e;
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
    // two slots a group
    return (size_t)2 * kGroups * std::min(sms, kAttendMaxCtas / kGroups) * 48 * (dim + 3);
}

}  // namespace lbv

// attend_tiles.cu -- attention of many new tokens over the paged cache
// (prompts' chunks, batches of drafts) on the 5th-generation tensor cores.
//
// The same sums as attend_rows.cu, over tiles of 128 rows (new token times
// query head of the group) and blocks of 128 keys.  Both products are
// tcgen05.mma with the rows as M: S = Q K^T from shared memory, then O += P V
// with P in tensor memory, where it replaces the fp32 S it came from.
//   * Two streams run side by side so that the tensor cores work on one while
//     the other's 128 threads (one row each) take its softmax: each has its
//     own S/P and O columns in tensor memory.  An item of more than 128 rows
//     gives the streams two row tiles that share every block of keys; a smaller
//     one gives them its even and its odd blocks and adds the two results.
//   * A copy warp fills a ring of 128-byte-swizzled slots, K and V of a block in
//     turn, by TMA; another warp issues the MMAs; commits free the slots.
//   * A row's reference maximum moves only when it grew by more than 8 (see
//     attend_rows.cu); only then are its sums in tensor memory rescaled, by the
//     row's own thread.
//   * The blocks of the batch are divided evenly over one CTA per SM, as in
//     attend_rows.cu; a causal tile counts those that it sees.  The parts of a
//     divided item are added by a launch of their own (attend_join.cu).
//
// What bounds it (48 query over 8 key/value heads of 128, bf16): in long items the
// hand-over of S and P, with the tensor cores 70 % busy: 2048 tokens at the end of 16,384
// take 510 to 530 us, 1,460 to 1,520 TFLOP/s.  In short ones their ends, during which the
// tensor cores wait: code that runs once an item is fetched anew and takes some 25 clocks an
// instruction, where the block's loop takes 9; 16 requests of 1 to 600 tokens take 139 us,
// their operations at the same rate 84.  With few blocks the start: 5 us to the first
// scores and 5 more to fetch the block's code, some 20 KB; 8 tokens after 32,771 take
// 36 us, their keys and values 20.
#include "attend_common.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kKeys = 128;                       // keys per block
constexpr int kTile = 128;                       // rows per stream
constexpr int kRows = 2 * kTile;                 // rows per item
// Units of an item: its queries and results, a block of one row tile, a block of two;
// and the least share of a CTA.  A unit is 0.2 us of a long item.  (16 requests of 1 to
// 600 tokens, us: 16/3/4 141, these 139, 28/3/4 141, 24/4/4 143, 36/4/5 142; a prompt's
// chunk is the same within 1 %.  The least share: 40 small batches take 4 % less with 8 or
// 12 than with 24, 12 % less than with 48; 20 tokens over 3,943 keys 15.6 and 20.3 us.)
constexpr int kExtra = 24, kNarrow = 3, kWide = 4, kMinUnits = 12;
using Items = Shape<kRows, kKeys, kExtra, kNarrow, kWide, kTile>;
constexpr int kThreads = 384;                    // copies and MMAs, then the two streams
// Registers a thread after the split: 168 * 384 at launch = 88 * 128 + 208 * 256.
constexpr int kRegsControl = 88, kRegsStream = 208;

constexpr int kItems = 4;                        // items the roles may be apart

// What the roles need to know of an item.
struct alignas(16) Item {
    Request q;
    int r, row0, rows, head, lo, hi;
    int key0, nb;          // its first key and its blocks in this share; 0 blocks: no more items
    int slot0;             // ring slots used before it
    int c0, c1;            // CTAs that hold a part of it
    __device__ bool dual() const { return rows > kTile; }
    __device__ bool whole() const { return c0 == c1; }
};
static_assert(sizeof(Item) == 64, "ring entry");

template <int D>
struct Geo {
    static constexpr int HALF = kKeys * 128;                // 64 elements of 128 rows
    static constexpr int SLOT = (D / 64) * HALF;            // one block's K or V; one Q tile
    static constexpr int Q = 0;
    static constexpr int RING = 2 * SLOT;
    static constexpr int NSLOT = D == 128 ? 5 : 10;
    static constexpr int BARS = RING + NSLOT * SLOT;
    static constexpr int NBARS = 2 * NSLOT + 11 + 2 * kItems;
    static constexpr int STATS = (BARS + NBARS * 8 + 15) / 16 * 16;   // [2][128] m and sums of the streams
    static constexpr int RATIOS = STATS + 2 * kTile * 8;    // [2][128] exact over rounded sums
    static constexpr int ITEMS = RATIOS + 2 * kTile * 2;    // ring of items
    static constexpr int WORDS = ITEMS + kItems * 64;       // tensor-memory address
    static constexpr int START = STATS;                     // the share's begin, before the first statistics
    static constexpr int BYTES = WORDS + 16;
    static constexpr int PARTIAL = kRows * (D + 3);         // floats of one partial result
    // tensor memory columns
    static constexpr uint32_t S0 = 0, O0 = 256;             // S of stream s at S0 + 128 s
    static_assert(BARS % 8 == 0 && STATS % 16 == 0 && ITEMS % 16 == 0 && WORDS % 16 == 0, "alignment");
    static_assert(BYTES <= 227 * 1024 && sizeof(Start) <= 2 * kTile * 8, "shared memory");
};

// ---- tcgen05 ----

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&d)[32])
{
    uint32_t* r = reinterpret_cast<uint32_t*>(d);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&d)[16])
{
    uint32_t* r = reinterpret_cast<uint32_t*>(d);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16};\n" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]),
        "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// Four steps of 16 of the contracted dimension, D (+)= A B, issued by one elected
// lane of a converged warp: their operands stay in uniform registers that way (a
// single thread in a branch of its own took 85 cycles an MMA to issue them).
// `add` 0: the first step overwrites D.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred e, p;\n setp.ne.b32 p, %10, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, 1;\n}\n" ::"r"(d), "l"(a), "l"(a + 2),
        "l"(a + 4), "l"(a + 6), "l"(b), "l"(b + 2), "l"(b + 4), "l"(b + 6), "r"(idesc), "r"(add)
        : "memory");
}

// The same with A (P) in tensor memory and B (V) with its rows along the
// contracted dimension: 8 columns of A and 16 rows of B a step.
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred e, p;\n setp.ne.b32 p, %10, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, 1;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, 1;\n}\n" ::"r"(d), "r"(a),
        "r"(a + 8), "r"(a + 16), "r"(a + 24), "l"(b), "l"(b + 128), "l"(b + 256), "l"(b + 384),
        "r"(idesc), "r"(add)
        : "memory");
}

// Arrives on `bar` once every MMA the elected lane has issued is complete.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor in 128-byte-swizzled rows: 8-row groups 1024
// bytes apart; for an operand whose rows run along the contracted dimension (V),
// `lead` bytes between its 64-element column groups.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lead)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, fp32 sums, M = 128; bit 16: B is N-major.
template <int DT>
__host__ __device__ constexpr uint32_t idesc(int n, bool b_n_major)
{
    return (1u << 4) | ((uint32_t)(DT == LBV_BF16) << 7) | ((uint32_t)(DT == LBV_BF16) << 10) |
           ((uint32_t)b_n_major << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;\n"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// Stores row `row` of a request and kv head (zeros if it is not `in` the item) as
// row `trow` of a Q tile at `tile`, in the layout of the copies.
template <int D>
__device__ __forceinline__ void store_q(const AttendParams& p, int q0, int kv_head, int row, bool in,
                                        unsigned char* tile, int trow)
{
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const int i = token_of(p, row);
    const uint16_t* src = p.q + (int64_t)(q0 + i) * p.q_token +
                          (int64_t)(kv_head * p.group + row - i * p.group) * p.q_head;
    uint4 v[D / 8];
#pragma unroll
    for (int ch = 0; ch < D / 8; ++ch)
        v[ch] = make_uint4(0u, 0u, 0u, 0u);
    if (in && p.scale_log2 != 0.f) {
        if (p.q_wide) {                              // all loads in flight before the first store
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch)
                v[ch] = __ldg(reinterpret_cast<const uint4*>(src) + ch);
        } else {
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch) {
                uint32_t e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    e[k] = (uint32_t)src[ch * 8 + 2 * k] | ((uint32_t)src[ch * 8 + 2 * k + 1] << 16);
                v[ch] = make_uint4(e[0], e[1], e[2], e[3]);
            }
        }
    }
    unsigned char* dst = tile + trow * 128;
#pragma unroll
    for (int ch = 0; ch < D / 8; ++ch) {
        v[ch].x ^= flip, v[ch].y ^= flip, v[ch].z ^= flip, v[ch].w ^= flip;
        *reinterpret_cast<uint4*>(dst + (ch >> 3) * Geo<D>::HALF + (((ch & 7) ^ (trow & 7)) << 4)) = v[ch];
    }
    fence_proxy_async_smem();
}

// The same by asynchronous copies, for aligned rows and a scale of 0 or more; the
// thread waits for them later.
template <int D>
__device__ __forceinline__ void fetch_q(const AttendParams& p, int q0, int kv_head, int row, bool in,
                                        uint32_t tile, int trow)
{
    const int i = token_of(p, row);
    const uint16_t* src = in ? p.q + (int64_t)(q0 + i) * p.q_token +
                                   (int64_t)(kv_head * p.group + row - i * p.group) * p.q_head
                             : p.q;
    const uint32_t bytes = in && p.scale_log2 != 0.f ? 16u : 0u;         // the rest is filled with zeros
    const uint32_t dst = tile + trow * 128;
#pragma unroll
    for (int ch = 0; ch < D / 8; ++ch)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                         dst + (ch >> 3) * Geo<D>::HALF + (((ch & 7) ^ (trow & 7)) << 4)),
                     "l"(src + (bytes ? ch * 8 : 0)), "r"(bytes)
                     : "memory");
}

template <int DT, int D>
__global__ void __launch_bounds__(kThreads, 1)
    lbv_attend_tiles_kernel(const __grid_constant__ AttendParams p,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap)
{
    using G = Geo<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem + G::WORDS);
    auto bar = [&](int i) { return sbase + G::BARS + i * 8; };
    auto full = [&](int i) { return bar(i); };
    auto empty = [&](int i) { return bar(G::NSLOT + i); };
    const uint32_t q_full = bar(2 * G::NSLOT);                       // both Q tiles are stored
    auto s_full = [&](int s) { return bar(2 * G::NSLOT + 1 + s); };  // S of stream s is complete
    auto o_done = [&](int s) { return bar(2 * G::NSLOT + 3 + s); };  // O has the block
    auto p_full = [&](int s, int half) { return bar(2 * G::NSLOT + 5 + 2 * s + half); };  // P replaced S
    auto item_full = [&](int i) { return bar(2 * G::NSLOT + 9 + i % kItems); };
    auto item_empty = [&](int i) { return bar(2 * G::NSLOT + 9 + kItems + i % kItems); };
    const uint32_t mmas_done = bar(2 * G::NSLOT + 9 + 2 * kItems);   // every MMA of the CTA
    const uint32_t together = bar(2 * G::NSLOT + 10 + 2 * kItems);   // both streams have come as far
    const Item* items = reinterpret_cast<const Item*>(smem + G::ITEMS);

    if (tid == 0) {
        for (int i = 0; i < G::NSLOT; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(q_full, 8);
        mbar_init(mmas_done, 1);
        mbar_init(together, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s, 0), 4);
            mbar_init(p_full(s, 1), 4);
            mbar_init(o_done(s), 1);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full(i), 1);
            mbar_init(item_empty(i), 10);                // copies, MMAs, eight warps of the streams
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    bool ok = true;
    after_previous();
    if (tid == 128)
        static_cast<JoinItem*>(p.items)[blockIdx.x].rows = 0;

    // After a wait that ran out, `ok` false, a thread waits for nothing more, goes on to its
    // item's end and leaves there with its warp.  Warps meet at bounded waits alone, so
    // that those it leaves behind run out too.  (The streams at a hardware barrier in place
    // of `together`: 137 us for the 139 above, and no end if one of them left.)
    auto wait = [&](uint32_t b, uint32_t parity) {
        if (ok)
            ok = mbar_wait(b, parity, p.wait_limit);
    };
    // item i of the share, as the scheduler wrote it, for a whole warp; valid if `ok`
    auto item_at = [&](int i) -> const Item& {
        wait(item_full(i), (uint32_t)((i / kItems) & 1));
        ok = __all_sync(0xffffffffu, ok);
        return items[i % kItems];
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsControl));
        if (warp == 0) {
            // ---- copies: K and V of each block in turn ----
            if (lane == 0) {
                prefetch_map(&kmap);
                prefetch_map(&vmap);
            }
            const int slots = min(64, 1 << p.kv.page_shift);         // rows of a box
            const int boxes = kKeys / slots;
            int n = 0;                                               // slots asked for
            for (int it = 0;; ++it) {
                const Item& w = item_at(it);
                if (!ok || w.nb == 0)
                    break;
                const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
                for (int i = 0; i < 2 * w.nb; ++i) {
                    const int st = n % G::NSLOT, k0 = w.key0 + (i >> 1) * kKeys;
                    // read, and its last copy landed (see attend_rows.cu)
                    if (n >= G::NSLOT) {
                        wait(empty(st), (uint32_t)((n / G::NSLOT - 1) & 1));
                        wait(full(st), (uint32_t)((n / G::NSLOT - 1) & 1));
                    }
                    ok = __all_sync(0xffffffffu, ok && ((unsigned)n < p.first_copies || blockIdx.x > 0));
                    if (!ok)
                        break;
                    ++n;
                    if (lane == 0)
                        mbar_expect_tx(full(st), G::SLOT);
                    __syncwarp();
                    for (int b = lane; b < boxes * (D / 64); b += 32) {
                        const int piece = b % boxes, half = b / boxes;
                        const int key = k0 + piece * slots;
                        int page = -1;                               // fills zeros
                        if (key < w.hi && key + slots > w.lo)
                            page = table[key >> p.kv.page_shift];
                        tma_box(sbase + G::RING + st * G::SLOT + half * G::HALF + piece * slots * 128,
                                (i & 1) ? &vmap : &kmap, half * 64,
                                key & ((1 << p.kv.page_shift) - 1), w.head, page, full(st));
                    }
                }
                __syncwarp();                                        // every lane has read the item
                if (lane == 0)
                    mbar_arrive(item_empty(it));
            }
            // the copies land before shared memory goes away, also after a wait that ran
            // out, and so do the commits that free their slots
            for (int i = 0; i < G::NSLOT; ++i)
                if (n - 1 - i >= 0 && !mbar_wait(full((n - 1 - i) % G::NSLOT),
                                                 (uint32_t)(((n - 1 - i) / G::NSLOT) & 1), p.wait_limit))
                    ok = false;
            for (int i = 0; i < G::NSLOT; ++i)
                if (n - 1 - i >= 0)
                    wait(empty((n - 1 - i) % G::NSLOT), (uint32_t)(((n - 1 - i) / G::NSLOT) & 1));
        } else if (warp == 1) {
            // ---- MMAs ----
            constexpr uint32_t id_s = idesc<DT>(kKeys, false), id_o = idesc<DT>(D, true);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            uint32_t n = 0, np0 = 0, np1 = 0;            // ring slots, blocks of each stream so far
            for (int it = 0;; ++it) {
                const Item& w = item_at(it);
                const int nb = __shfl_sync(0xffffffffu, w.nb, 0);
                const bool dual = __shfl_sync(0xffffffffu, w.rows, 0) > kTile;
                if (!ok || nb == 0)
                    break;
                wait(q_full, (uint32_t)(it & 1));
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(item_empty(it));
                __syncwarp();
                tc_fence_after();
                // K of block j is slot 2 j from the item's first, V the one after it
                auto arrived = [&](uint32_t i) {
                    wait(full(i % G::NSLOT), (i / G::NSLOT) & 1);
                    __syncwarp();
                };
                auto release = [&](uint32_t i) { commit(empty(i % G::NSLOT)); };
                auto score = [&](int s, int tile, uint32_t i) {      // S_s = Q_tile K^T
                    const uint64_t a = desc128(sbase + G::Q + tile * G::SLOT, 0);
                    const uint64_t b = desc128(sbase + G::RING + (i % G::NSLOT) * G::SLOT, 0);
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        mma4_ss(tm + G::S0 + s * 128, a + h * (G::HALF >> 4), b + h * (G::HALF >> 4), id_s,
                                h > 0);
                    commit(s_full(s));
                };
                auto value = [&](int s, uint32_t& np, uint32_t i, bool add) {    // O_s += P_s V
                    const uint64_t b = desc128(sbase + G::RING + (i % G::NSLOT) * G::SLOT, G::HALF);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {                    // 64 keys of P at a time
                        wait(p_full(s, h), np & 1);
                        __syncwarp();
                        tc_fence_after();
                        mma4_ts(tm + G::O0 + s * 128, tm + G::S0 + s * 128 + h * 32, b + h * 512, id_o,
                                add || h > 0);
                    }
                    ++np;
                    commit(o_done(s));
                };
                if (dual) {
                    arrived(n);
                    score(0, 0, n);
                    score(1, 1, n);
                    release(n);
                    for (int j = 0; j < nb; ++j, n += 2) {
                        arrived(n + 1);
                        if (j + 1 < nb)
                            arrived(n + 2);
                        value(0, np0, n + 1, j > 0);
                        if (j + 1 < nb)
                            score(0, 0, n + 2);
                        value(1, np1, n + 1, j > 0);
                        release(n + 1);
                        if (j + 1 < nb) {
                            score(1, 1, n + 2);
                            release(n + 2);
                        }
                    }
                } else {
                    for (int j = 0; j < 2 && j < nb; ++j) {
                        arrived(n + 2 * j);
                        score(j, 0, n + 2 * j);
                        release(n + 2 * j);
                    }
                    for (int j = 0; j < nb; ++j, n += 2) {
                        arrived(n + 1);
                        if (j & 1)
                            value(1, np1, n + 1, j > 1);
                        else
                            value(0, np0, n + 1, j > 1);
                        release(n + 1);
                        if (j + 2 < nb) {
                            arrived(n + 4);
                            score(j & 1, 0, n + 4);
                            release(n + 4);
                        }
                    }
                }
            }
            // the last MMAs end before tensor memory goes away, also after a wait that ran out
            __syncwarp();
            commit(mmas_done);
            if (!mbar_wait(mmas_done, 0, p.wait_limit))
                ok = false;
        } else if (warp == 2) {
            // ---- the share's items ----
            Start& start = *reinterpret_cast<Start*>(smem + G::START);
            find_start<Items>(p, lane, gridDim.x, kMinUnits, blockIdx.x, &start);
            __syncwarp();
            Item* out = reinterpret_cast<Item*>(smem + G::ITEMS);
            if ((int)blockIdx.x >= start.ctas) {             // fewer units than CTAs
                if (lane == 0) {
                    out[0].nb = 0;
                    mbar_arrive(item_full(0));
                }
            } else {
                Walk<Items> w(p, start, blockIdx.x);
                int slot0 = 0;
                for (int it = 0;; ++it) {
                    const bool more = w.next();
                    if (it >= kItems)
                        wait(item_empty(it), (uint32_t)((it / kItems - 1) & 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)                                 // its place is still read
                        break;
                    if (lane == 0) {
                        const int nb = more ? w.b_last - w.b_first : 0;
                        out[it % kItems] = {w.q, w.r, w.x.row0, w.x.rows, w.head, w.x.lo, w.x.hi,
                                            w.key0(w.b_first), nb, slot0, w.first_cta(), w.last_cta()};
                        mbar_arrive(item_full(it));          // releases the stores
                        slot0 += 2 * nb;
                    }
                    // its queries are on the way before the streams ask for them
                    if (more)
                        for (int i = lane; i < w.x.rows * (D / 64); i += 32) {
                            const int row = w.x.row0 + i / (D / 64), tok = token_of(p, row);
                            prefetch_l2(p.q + (int64_t)(w.q.q0 + tok) * p.q_token +
                                        (int64_t)(w.head * p.group + row - tok * p.group) * p.q_head +
                                        i % (D / 64) * 64);
                        }
                    if (!more)
                        break;
                }
            }
        }
        __syncwarp();
    } else {
        // ---- the streams: one row a thread ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsStream));
        const int s = (warp >> 2) - 1;                               // stream
        const int trow = tid & 127;                                  // row within the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + G::S0 + s * 128, o_at = tmem + lanes + G::O0;
        float2* stats = reinterpret_cast<float2*>(smem + G::STATS);
        int16_t* ratios = reinterpret_cast<int16_t*>(smem + G::RATIOS);
        // scores are c times Q's: a negative scale negates Q, a zero one clears it
        const float c = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
        int done = 0;                    // blocks of this stream so far
        int met = 0;                     // meetings of the two streams so far
        auto meet = [&] {
            __syncwarp();
            if (lane == 0)
                mbar_arrive(together);
            wait(together, (uint32_t)(met++ & 1));
        };
        // Stores this thread's row of an item's Q.  The MMAs that read the Q tiles of
        // the item before are complete: their scores have been read.
        auto enter = [&](const Item& w) {
            const bool dual = w.dual();
            const int item_row = dual ? s * kTile + trow : trow;
            const bool in = item_row < w.rows;
            if (dual || s == 0)
                store_q<D>(p, w.q.q0, w.head, w.row0 + item_row, in, smem + G::Q + s * G::SLOT, trow);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full);
        };
        bool more = item_at(0).nb > 0 && ok;
        if (more)
            enter(items[0]);
        for (int it = 0; more; ++it) {
            const Item& w = items[it % kItems];
            const bool dual = w.dual();
            const int nb = w.nb;
            const int item_row = dual ? s * kTile + trow : trow;
            float m = -INFINITY;
            // sums of the probabilities as they enter the product, and exact
            float2 l = make_float2(0.f, 0.f), x = make_float2(0.f, 0.f);
            int mine = 0;                                            // blocks of this item
            bool fetched = false;                                    // the next item's queries are on the way
            {
                const bool in = item_row < w.rows;
                const int i = token_of(p, w.row0 + item_row);
                const int pos = in ? w.q.first + i : INT_MIN / 2;
                const uint64_t word = in && p.tree ? p.tree[w.q.q0 + i] : 0;
                // keys at `open_hi` and past, or below `open_lo`, are hidden from some
                // row of the tile
                const int r0 = w.row0 + (dual ? s * kTile : 0);
                const int r1 = min(r0 + kTile, w.row0 + w.rows) - 1;
                const int open_hi = p.tree ? min(w.q.keys, w.q.first)
                                           : min(w.q.keys, w.q.first + token_of(p, r0) + 1);
                const int open_lo = p.window > 0 ? w.q.first + token_of(p, r1) - p.window + 1 : 0;
                const bool idle = r0 + (warp & 3) * 32 > r1;         // no row in this warp
                for (int j = dual ? 0 : s; j < nb; j += dual ? 1 : 2, ++mine, ++done) {
                    const int k0 = w.key0 + j * kKeys;
                    wait(s_full(s), (uint32_t)(done & 1));
                    tc_fence_after();
                    // the last scores of two row tiles: this stream's Q is free, and the copy
                    // of the next takes as long as this block
                    if (dual && j + 1 == nb && p.q_wide && p.scale_log2 >= 0.f) {
                        const Item& v = item_at(it + 1);
                        if (v.nb > 0 && ok && (v.dual() || s == 0)) {
                            const int row = (v.dual() ? s * kTile : 0) + trow;
                            fetch_q<D>(p, v.q.q0, v.head, v.row0 + row, row < v.rows,
                                       sbase + G::Q + s * G::SLOT, trow);
                            fetched = true;
                        }
                    }
                    // slots past the context may hold anything: NaN times 0 is not 0
                    if (k0 + kKeys > w.q.keys) {
                        const int v = w.slot0 + 2 * j + 1;
                        wait(full(v % G::NSLOT), (uint32_t)((v / G::NSLOT) & 1));
                        if (k0 + trow >= w.q.keys) {
                            unsigned char* z = smem + G::RING + (v % G::NSLOT) * G::SLOT + trow * 128;
#pragma unroll
                            for (int e = 0; e < D / 8; ++e)
                                *reinterpret_cast<uint4*>(z + (e >> 3) * G::HALF + ((e & 7) << 4)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    float t[4][32];
                    if (!idle) {
                        // masked scores are overwritten in place (rare, so short code)
                        if (k0 + kKeys > open_hi || k0 < open_lo) {
#pragma unroll 1
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t see = seen32(p, w.q, pos, word, k0 + (e & ~1) * 16) >> (e & 1) * 16;
                                float u[16];
                                uint32_t r[16];
                                tmem_ld16(s_at + e * 16, u);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    r[k] = (see >> k) & 1u ? __float_as_uint(u[k]) : 0xFF800000u;
                                tmem_st16(s_at + e * 16, r);
                            }
                            tmem_wait_st();
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            tmem_ld32(s_at + e * 32, t[e]);
                        tmem_wait_ld();
                    }
                    // P of 32 keys and its sum, for the reference m
                    uint32_t r[16];
                    float2 part;
                    auto exps = [&](int e) {
                        const float ref = m == -INFINITY ? 0.f : -m;
                        part = make_float2(0.f, 0.f);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float2 v = fma2(make_float2(t[e][2 * k], t[e][2 * k + 1]), make_float2(c, c),
                                            make_float2(ref, ref));
                            v.x = ex2(v.x), v.y = ex2(v.y);
                            part = add2(part, v);
                            r[k] = pack2<DT>(v.x, v.y);
                        }
                    };
                    float2 block = make_float2(0.f, 0.f);            // the block's sum
                    bool heavy = false;                              // one key is half of the sum or more
                    if (!idle) {
                        // the first 32 keys with the reference as it is, while the block's
                        // maximum is found; once more if that moves the reference
                        exps(0);
                        float tops[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            tops[e] = fmaxf(t[e][0], t[e][1]);
#pragma unroll
                            for (int k = 2; k < 32; k += 2)
                                tops[e] = fmaxf(tops[e], fmaxf(t[e][k], t[e][k + 1]));
                        }
                        const float top = c * fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                        const bool moved = top > m + 8.f;            // also from -inf
                        if (__any_sync(0xffffffffu, moved)) {
                            const float f = moved ? ex2(m - top) : 1.f;
                            m = moved ? top : m;
                            l.x *= f, l.y *= f, x.x *= f, x.y *= f;
                            if (mine > 0) {
                                wait(o_done(s), (uint32_t)((done - 1) & 1));
                                tc_fence_after();
#pragma unroll 1
                                for (int e = 0; e < D / 16; ++e) {
                                    float o[16];
                                    tmem_ld16(o_at + s * 128 + e * 16, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        r[k] = __float_as_uint(o[k] * f);
                                    tmem_st16(o_at + s * 128 + e * 16, r);
                                }
                            }
                            exps(0);
                        }
                        heavy = 2.f * ex2(top - m) >= x.x + x.y;
                        block = part;
                        tmem_st16(s_at, r);
                        exps(1);
                        block = add2(block, part);
                        tmem_st16(s_at + 16, r);
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_full(s, 0));
                    if (!idle) {
                        const bool few = __any_sync(0xffffffffu, heavy);
#pragma unroll
                        for (int e = 2; e < 4; ++e) {
                            exps(e);
                            block = add2(block, part);
                            tmem_st16(s_at + e * 16, r);
                        }
                        tmem_wait_st();
                        x = add2(x, block);
                        // What V is multiplied with is rounded: a row that few keys dominate is
                        // divided by the sum of the rounded values, so that it gets those keys'
                        // values; elsewhere the roundings cancel.
                        if (few) {
                            block = make_float2(0.f, 0.f);
#pragma unroll 1
                            for (int e = 0; e < 4; ++e) {
                                float v[16];
                                tmem_ld16(s_at + e * 16, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    block = add2(block, unpack2<DT>(__float_as_uint(v[k])));
                            }
                        }
                        l = add2(l, block);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(p_full(s, 1));
                }
            }

            // ---- the item's result, while the next item's first scores are computed ----
            if (!dual)                                   // both streams read tile 0, which stream 0 stores
                meet();
            more = item_at(it + 1).nb > 0 && ok;
            if (fetched) {
                asm volatile("cp.async.wait_all;\n" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full);
            } else if (more) {
                enter(items[(it + 1) % kItems]);
            }
            if (mine > 0)
                wait(o_done(s), (uint32_t)((done - 1) & 1));
            float sum = l.x + l.y, exact = x.x + x.y;
            float f0 = 1.f, f1 = 0.f;                    // factors of this row in O_0 and O_1
            if (!dual) {
                stats[s * kTile + trow] = make_float2(m, sum);
                // the sums differ by less than 2^-8 of them, kept to 2^-23
                ratios[s * kTile + trow] =
                    sum > 0.f ? (int16_t)max(-32767, min(32767, __float2int_rn((exact / sum - 1.f) * 4194304.f)))
                              : (int16_t)0;
                tc_fence_before();
                meet();
                const float2 a = stats[trow], b = stats[kTile + trow];
                m = fmaxf(a.x, b.x);
                f0 = a.x == -INFINITY ? 0.f : ex2(a.x - m);
                f1 = b.x == -INFINITY ? 0.f : ex2(b.x - m);
                sum = f0 * a.y + f1 * b.y;
                exact = f0 * a.y * (1.f + ratios[trow] * (1.f / 4194304.f)) +
                        f1 * b.y * (1.f + ratios[kTile + trow] * (1.f / 4194304.f));
            }
            tc_fence_after();
            const bool in = item_row < w.rows, whole = w.whole();
            const int row = w.row0 + item_row, i = token_of(p, row);
            const int64_t tok = w.q.q0 + i;
            const int head = w.head * p.group + row - i * p.group;
            float* slot = p.partial + (size_t)(2 * blockIdx.x + (w.c0 == (int)blockIdx.x)) * G::PARTIAL;
            // dual: all columns of the row; else the stream's half of them
            const int e0 = dual ? 0 : s * (D / 64), e1 = dual ? D / 32 : (s + 1) * (D / 64);
            // (the quotient is rounded to 16 bits: an approximate reciprocal, off by 2^-23, will do)
            const float f = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
#pragma unroll 1
            for (int e = e0; e < e1; ++e) {
                float o[32];
                tmem_ld32(o_at + (dual ? s * 128 : 0) + e * 32, o);
                if (!dual) {
                    float o1[32];
                    tmem_ld32(o_at + 128 + e * 32, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 32; ++k)         // what was never written counts as 0
                        o[k] = (f0 > 0.f ? f0 * o[k] : 0.f) + (f1 > 0.f ? f1 * o1[k] : 0.f);
                } else {
                    tmem_wait_ld();
                }
                if (in && whole) {
                    uint32_t r[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        r[k] = sum == 0.f ? 0u : pack2<DT>(o[2 * k] * f, o[2 * k + 1] * f);
                    store_row<32>(p.out + tok * p.out_token + (int64_t)head * p.out_head + e * 32, r);
                } else if (in) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t r[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            r[i] = sum == 0.f ? 0u : __float_as_uint(o[8 * k + i]);
                        store32(slot + item_row * D + e * 32 + 8 * k, r);
                    }
                }
            }
            if (in && (dual || s == 0)) {
                if (whole && p.lse) {
                    p.lse[tok * p.heads + head] = lse_of(m, exact);
                } else if (!whole) {
                    slot[kRows * D + item_row] = m;
                    slot[kRows * (D + 1) + item_row] = sum;
                    slot[kRows * (D + 2) + item_row] = exact;
                }
            }
            if (!whole && tid == 128 && w.c0 == (int)blockIdx.x)
                static_cast<JoinItem*>(p.items)[w.c0] = {w.q.q0, w.row0, w.rows, w.head,
                                                         w.c1 - w.c0 + 1};
            tc_fence_before();
            if (!dual)                                   // both streams are done reading O and the statistics
                meet();
            __syncwarp();                                // every lane has read the item
            if (lane == 0)
                mbar_arrive(item_empty(it));
        }
    }
    if (!ok)
        atomicOr(p.status, 1u);
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }
}

template <int DT, int D>
cudaError_t launch(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                   cudaStream_t st)
{
    auto kernel = lbv_attend_tiles_kernel<DT, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Geo<D>::BYTES);
    if (e != cudaSuccess)
        return e;
    const int ctas = sms < kAttendMaxCtas ? sms : kAttendMaxCtas;
    e = launch_after(kernel, dim3((unsigned)ctas), kThreads, Geo<D>::BYTES, st, p, kmap, vmap);
    return e == cudaSuccess ? launch_attend_join(p, (lbv_dtype)DT, kRows, ctas, st) : e;
}

}  // namespace

cudaError_t launch_attend_tiles(const AttendParams& p, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, lbv_dtype dt, int sms, cudaStream_t st)
{
    if (dt == LBV_F16)
        return p.kv.dim == 128 ? launch<LBV_F16, 128>(p, kmap, vmap, sms, st)
                               : launch<LBV_F16, 64>(p, kmap, vmap, sms, st);
    return p.kv.dim == 128 ? launch<LBV_BF16, 128>(p, kmap, vmap, sms, st)
                           : launch<LBV_BF16, 64>(p, kmap, vmap, sms, st);
}

size_t attend_tiles_partial_floats(int dim, int sms)
{
    return (size_t)2 * (sms < kAttendMaxCtas ? sms : kAttendMaxCtas) * kRows * (dim + 3);
}

}  // namespace lbv

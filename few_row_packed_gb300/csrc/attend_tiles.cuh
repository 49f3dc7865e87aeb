// attend_tiles.cuh -- attention of many new tokens over the paged cache
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
//   * Over a cache of 4 bits two warps copy pieces of codes and scales, and four more
//     expand them and store the slots' rows.
//   * The blocks of the batch are divided evenly over one CTA per SM, as in
//     attend_rows.cu; a causal tile counts those that it sees.  The parts of a
//     divided item are added by a launch of their own (attend_join.cu).
//
// What bounds it (48 query over 8 key/value heads of 128, bf16): in long items the
// hand-over of S and P, with the tensor cores 70 % busy: 2048 tokens at the end of 16,384
// take 480 to 520 us, 1,490 to 1,600 TFLOP/s, by the clocks (a long series of calls meets the
// power limit).  In short ones their ends, during which the
// tensor cores wait: code that runs once an item is fetched anew and takes some 25 clocks an
// instruction, where the block's loop takes 9; 16 requests of 1 to 600 tokens take 135 us,
// their operations at the same rate 77.  With few blocks the start: 5 us to the first
// scores and 5 more to fetch the block's code, some 20 KB; 8 tokens after 32,771 take
// 36 us, their keys and values 20.
//
// Over a cache of 4 bits the four warps that expand: of 1,500 clocks a slot they spend 790 to
// expand and store a thread's 128 elements, 75 in the fence before the MMAs read them, and the
// rest waiting for codes and for places.  With two row tiles a block's products take nearly as long:
// 2048 tokens at the end of 16,384 take 560 to 600 us.  With one they do
// not: 32 requests of 8 tokens over 7,000 keys 142 us, from 16 bits 159.  Eight warps, keys and
// values apart, leave the streams 168 registers or less, whose spills cost more than is won: 603
// to 670 us and 157 to 163.
#pragma once

#include "attend_common.cuh"
#include "attend_tc.cuh"
#include "kv4.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kKeys = 128;                       // keys per block
constexpr int kTile = 128;                       // rows per stream
constexpr int kRows = 2 * kTile;                 // rows per item
// Units of an item: its queries and results, a block of one row tile, a block of two;
// and the least share of a CTA.  A unit is 0.2 us of a long item.  (16 requests of 1 to
// 600 tokens: 16/3/4 and 28/3/4 take 1.5 % longer, 24/4/4 3, 36/4/5 2; a prompt's
// chunk is the same within 1 %.  The least share: 40 small batches take 4 % less with 8 or
// 12 than with 24, 12 % less than with 48; 20 tokens over 3,943 keys 15.6 and 20.3 us.)
// Over 4 bits a block takes as long to expand for one row tile as for two: 16/4/4 is 1 to 5 %
// faster there than 24/3/4 (64 requests of 4 to 16 tokens 122 us and 128, the 16 above 167 and 170);
// 12 and 24 are between.
constexpr int kMinUnits = 12;
template <bool KV4>
using Items = Shape<kRows, kKeys, KV4 ? 16 : 24, KV4 ? 4 : 3, 4, kTile>;
// Warps: copies and MMAs, then the two streams; over a cache of 4 bits four more, which expand what
// the copies bring into the slots.
template <bool KV4>
struct Roles {
    static constexpr int THREADS = KV4 ? 512 : 384;
    // registers a thread after the split: 168 * 384 at launch = 88 * 128 + 208 * 256, and
    // 128 * 512 = (80 + 48) * 128 + 192 * 256 (64 to expand and 184 for the streams: 1 to 4 %
    // longer; 72 + 56: 2 %; 64 + 48 and 200: 3 to 5 %)
    static constexpr int CONTROL = KV4 ? 80 : 88, STREAM = KV4 ? 192 : 208, EXPAND = 48;
    // who fills a slot, and who reads an item (copies, of 4 bits by two warps, MMAs, eight warps
    // of the streams, and those that expand)
    static constexpr int FILLERS = KV4 ? 4 : 1, READERS = KV4 ? 15 : 10;
};

constexpr int kItems = 4;                        // items the roles may be apart

// What the roles need to know of an item.
struct alignas(16) Item {
    int q0, first, keys;   // of its request
    int r, row0, rows, head, lo, hi;
    int key0, nb;          // its first key and its blocks in this share; 0 blocks: no more items
    int skip;              // keys left out before block `jump` (behind the sinks)
    int jump;
    int slot0;             // ring slots used before it
    int c0, c1;            // CTAs that hold a part of it
    __device__ int key_of(int j) const { return key0 + j * kKeys + (j >= jump ? skip : 0); }
    __device__ bool dual() const { return rows > kTile; }
    __device__ bool whole() const { return c0 == c1; }
};
static_assert(sizeof(Item) == 64, "ring entry");

template <int D, bool KV4>
struct Geo {
    static constexpr int HALF = kKeys * 128;                // 64 elements of 128 rows
    static constexpr int SLOT = (D / 64) * HALF;            // one block's K or V; one Q tile
    static constexpr int Q = 0;
    static constexpr int RING = 2 * SLOT;
    static constexpr int NSLOT = (D == 128 ? 5 : 10) - (KV4 ? 128 / D : 0);
    // 4 bits: a ring of a block's keys or values as they are held, codes and then scales (three
    // of them beside four slots; six beside three slots take the same time within 3 %)
    static constexpr int HELD = RING + NSLOT * SLOT;
    static constexpr int CODES = kKeys * 32 * (D / 64), HSLOT = kKeys * 36 * (D / 64);
    static constexpr int NHELD = KV4 ? (D == 128 ? 3 : 6) : 0;
    static constexpr int BARS = HELD + NHELD * HSLOT;
    static constexpr int NBARS = 2 * NSLOT + 11 + 2 * kItems + 2 * NHELD;
    static constexpr int THERE = BARS + NBARS * 8;          // their chunks that exist
    static constexpr int STATS = (THERE + NHELD * 4 + 15) / 16 * 16;   // [2][128] m and sums of the streams
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
        *reinterpret_cast<uint4*>(dst + (ch >> 3) * kKeys * 128 + (((ch & 7) ^ (trow & 7)) << 4)) = v[ch];
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
                         dst + (ch >> 3) * kKeys * 128 + (((ch & 7) ^ (trow & 7)) << 4)),
                     "l"(src + (bytes ? ch * 8 : 0)), "r"(bytes)
                     : "memory");
}

template <int DT, int D, bool KV4>
__global__ void __launch_bounds__(Roles<KV4>::THREADS, 1)
    lbv_attend_tiles_kernel(const __grid_constant__ AttendParams p,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap)
{
    using G = Geo<D, KV4>;
    using R = Roles<KV4>;
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
    auto held_full = [&](int i) { return bar(2 * G::NSLOT + 11 + 2 * kItems + i); };
    auto held_empty = [&](int i) { return bar(2 * G::NSLOT + 11 + 2 * kItems + G::NHELD + i); };
    const Item* items = reinterpret_cast<const Item*>(smem + G::ITEMS);

    if (tid == 0) {
        for (int i = 0; i < G::NSLOT; ++i) {
            mbar_init(full(i), R::FILLERS);
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
        for (int i = 0; i < G::NHELD; ++i) {
            mbar_init(held_full(i), 1);
            mbar_init(held_empty(i), 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full(i), 1);
            mbar_init(item_empty(i), R::READERS);
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
    // of `together`: 1.5 % less for the 16 requests above, and no end if one of them left.)
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R::CONTROL));
        if (KV4 && (warp == 0 || warp == 3)) {
            // ---- copies as the rows are held: K of each block by one warp, V by the other; lanes
            // 2 i and 2 i + 1 have the codes and the scales of chunk i.  (A lane's copy takes its
            // warp some 40 clocks to issue: 32 requests of 8 tokens over 7,000 keys take 209 us with
            // pages of 16 slots and one warp, 147 with two; heads of 64, pages of 64, 132 and 103.) ----
            const int cs = kv4::chunk_shift(p.kv), chunk0 = (lane >> 1) << cs;
            const int64_t page_bytes = kv4::page_bytes(p.kv);
            const uint32_t size = lane & 1 ? 4 * (D / 64) << cs : 32 * (D / 64) << cs;
            const int v = warp == 3;
            int n = v;                                               // the next copy
            for (int it = 0;; ++it) {
                const Item& w = item_at(it);
                if (!ok || w.nb == 0)
                    break;
                const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
                const uint8_t* base = kv4::chunk(p.kv, 0, w.head, 0) + (lane & 1 ? D << cs : 0);
                auto page_of = [&](int j) {                          // of the chunk in block j, -1: zeros
                    const int key = w.key_of(j) + chunk0;
                    return j < w.nb && chunk0 < kKeys && wanted(p, w.lo, w.hi, key, 1 << cs)
                               ? table[key >> p.kv.page_shift]
                               : -1;
                };
                int next = page_of(0);
                for (int b = 0; b < w.nb; ++b) {
                    const int st = n % max(G::NHELD, 1), k0 = w.key_of(b), page = next;
                    next = page_of(b + 1);
                    // read, and its last copy landed (see attend_rows.cu).  In a ring of an odd length
                    // that copy was the other warp's.  This warp's copy before had waited for the
                    // reading of a later one than the place's last but one, so the parity cannot
                    // mean that one.
                    if (n >= G::NHELD) {
                        wait(held_empty(st), (uint32_t)((n / max(G::NHELD, 1) - 1) & 1));
                        wait(held_full(st), (uint32_t)((n / max(G::NHELD, 1) - 1) & 1));
                    }
                    ok = __all_sync(0xffffffffu, ok && ((unsigned)n < p.first_copies || blockIdx.x > 0));
                    if (!ok)
                        break;
                    n += 2;
                    const bool go = page >= 0 && page < p.kv.pages;
                    const unsigned there = __ballot_sync(0xffffffffu, go);
                    if (lane == 0) {
                        // all ones: every key of the block exists
                        const int chunks = __popc(there) / 2;
                        reinterpret_cast<uint32_t*>(smem + G::THERE)[st] =
                            chunks == kKeys >> cs && k0 + kKeys <= w.keys ? ~0u : there & 0x55555555u;
                        mbar_expect_tx(held_full(st), chunks * (36 * (D / 64) << cs));
                    }
                    __syncwarp();
                    if (go) {
                        const int s = (k0 + chunk0) & ((1 << p.kv.page_shift) - 1);
                        bulk_copy(sbase + G::HELD + st * G::HSLOT + (lane & 1 ? G::CODES : 0) + (lane >> 1) * size,
                                  base + page * page_bytes + (s >> cs) * (kv4::slot_bytes(D) << cs) + v * size,
                                  size, held_full(st));
                    }
                }
                __syncwarp();                                        // every lane has read the item
                if (lane == 0)
                    mbar_arrive(item_empty(it));
            }
            // the copies land before shared memory goes away, also after a wait that ran out: the
            // ring's last, or then this warp's own
            const int last = ok ? (n & ~1) - 1 : n - 2, step = ok ? 1 : 2;
            for (int i = last; i >= 0 && i > last - G::NHELD; i -= step)
                if (!mbar_wait(held_full(i % max(G::NHELD, 1)), (uint32_t)((i / max(G::NHELD, 1)) & 1), p.wait_limit))
                    ok = false;
        } else if (warp == 0) {
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
                    const int st = n % G::NSLOT, k0 = w.key_of(i >> 1);
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
                        if (wanted(p, w.lo, w.hi, key, slots))
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
            find_start<Items<KV4>>(p, lane, gridDim.x, kMinUnits, blockIdx.x, &start);
            __syncwarp();
            Item* out = reinterpret_cast<Item*>(smem + G::ITEMS);
            if ((int)blockIdx.x >= start.ctas) {             // fewer units than CTAs
                if (lane == 0) {
                    out[0].nb = 0;
                    mbar_arrive(item_full(0));
                }
            } else {
                Walk<Items<KV4>> w(p, start, blockIdx.x);
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
                        const bool split = w.b_first < w.x.near;     // sinks, then a window
                        out[it % kItems] = {w.q.q0, w.q.first, w.q.keys, w.r, w.x.row0, w.x.rows, w.head,
                                            w.x.lo, w.x.hi, w.key0(w.b_first), nb,
                                            split ? w.x.gap * kKeys : 0, w.x.near - w.b_first, slot0,
                                            w.first_cta(), w.last_cta()};
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
    } else if (KV4 && warp >= 12) {
        // ---- a cache of 4 bits: one key of a block a thread, its K and its V in turn ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R::EXPAND));
        const int row = tid & 127, cs = kv4::chunk_shift(p.kv), chunk = row >> cs;
        const int first = ((chunk * (D / 64) - chunk) << cs) + row;  // its first row of codes
        const uint32_t codes = sbase + G::HELD + first * 32, pairs = sbase + G::HELD + G::CODES + first * 4;
        // (the vector of codes goes first that leaves the lanes' banks apart)
        const int turn = (row >> 2) & 1;
        const uint32_t to = sbase + G::RING + row * 128 + (((row & 7) ^ (turn << 2)) << 4);
        const kv4::Constants constants = kv4::constants<DT>();
        int n = 0;                                                   // slots filled
        for (int it = 0;; ++it) {
            const Item& w = item_at(it);
            if (!ok || w.nb == 0)
                break;
            for (int i = 0; i < 2 * w.nb; ++i) {
                const int st = n % max(G::NHELD, 1), slot = n % G::NSLOT;
                wait(held_full(st), (uint32_t)((n / max(G::NHELD, 1)) & 1));
                const uint32_t at = st * G::HSLOT, there = load4(sbase + G::THERE + 4 * st);
                uint32_t held[D / 32][4], pair[D / 64];
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    load16((codes + at + (part * 32 << cs)) ^ (turn << 4), held[2 * part]);
                    load16((codes + at + (part * 32 << cs)) ^ ((turn ^ 1) << 4), held[2 * part + 1]);
                    pair[part] = load4(pairs + at + (part * 4 << cs));
                }
                // slots past the context hold anything
                if (there != ~0u && !(((there >> (2 * chunk)) & 1) && w.key_of(i >> 1) + row < w.keys)) {
#pragma unroll
                    for (int part = 0; part < D / 64; ++part)
                        pair[part] = 0;
                }
                if (n >= G::NSLOT)
                    wait(empty(slot), (uint32_t)((n / G::NSLOT - 1) & 1));
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                ++n;
                __syncwarp();                                        // every lane has read
                if (lane == 0)
                    mbar_arrive(held_empty(st));
#pragma unroll
                for (int part = 0; part < D / 64; ++part) {
                    const uint32_t sc = kv4::both_scales(pair[part]), bi = kv4::both_biases(pair[part]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t v[4];
                        kv4::expand<DT>(held[2 * part + (e >> 2)][e & 3], sc, bi, constants, v);
                        store16((to ^ (e << 4)) + slot * G::SLOT + part * G::HALF, v);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(full(slot));
            }
            __syncwarp();                                            // every lane has read the item
            if (lane == 0)
                mbar_arrive(item_empty(it));
        }
        // the commits that free the slots land before shared memory goes away
        for (int i = 0; i < G::NSLOT; ++i)
            if (n - 1 - i >= 0)
                wait(empty((n - 1 - i) % G::NSLOT), (uint32_t)(((n - 1 - i) / G::NSLOT) & 1));
    } else {
        // ---- the streams: one row a thread ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(R::STREAM));
        const int s = (warp >> 2) - 1;                               // stream
        const int trow = tid & 127;                                  // row within the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + G::S0 + s * 128, o_at = tmem + lanes + G::O0;
        float2* stats = reinterpret_cast<float2*>(smem + G::STATS);
        int16_t* ratios = reinterpret_cast<int16_t*>(smem + G::RATIOS);
        // scores are c0 times Q's: a negative scale negates Q, a zero one clears it
        const float c0 = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
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
                store_q<D>(p, w.q0, w.head, w.row0 + item_row, in, smem + G::Q + s * G::SLOT, trow);
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
            float m = -INFINITY, c = c0;                             // c: what the row's scores are multiplied by
            // sums of the probabilities as they enter the product, and exact
            float2 l = make_float2(0.f, 0.f), x = make_float2(0.f, 0.f);
            int mine = 0;                                            // blocks of this item
            bool fetched = false;                                    // the next item's queries are on the way
            {
                const bool in = item_row < w.rows;
                const int i = token_of(p, w.row0 + item_row);
                const int pos = in ? w.first + i : INT_MIN / 2;
                const uint64_t word = in && p.tree ? p.tree[w.q0 + i] : 0;
                // keys at `open_hi` and past, or below `open_lo`, are hidden from some
                // row of the tile
                const int r0 = w.row0 + (dual ? s * kTile : 0);
                const int r1 = min(r0 + kTile, w.row0 + w.rows) - 1;
                const int open_hi = p.tree ? min(w.keys, w.first)
                                           : min(w.keys, w.first + token_of(p, r0) + 1);
                const int open_lo = p.window > 0 ? w.first + token_of(p, r1) - p.window + 1 : 0;
                const bool idle = r0 + (warp & 3) * 32 > r1;         // no row in this warp
                for (int j = dual ? 0 : s; j < nb; j += dual ? 1 : 2, ++mine, ++done) {
                    const int k0 = w.key_of(j);
                    wait(s_full(s), (uint32_t)(done & 1));
                    tc_fence_after();
                    // the last scores of two row tiles: this stream's Q is free, and the copy
                    // of the next takes as long as this block
                    if (dual && j + 1 == nb && p.q_wide && p.scale_log2 >= 0.f) {
                        const Item& v = item_at(it + 1);
                        if (v.nb > 0 && ok && (v.dual() || s == 0)) {
                            const int row = (v.dual() ? s * kTile : 0) + trow;
                            fetch_q<D>(p, v.q0, v.head, v.row0 + row, row < v.rows,
                                       sbase + G::Q + s * G::SLOT, trow);
                            fetched = true;
                        }
                    }
                    // slots past the context may hold anything: NaN times 0 is not 0 (expanded ones
                    // hold zeros)
                    if (!KV4 && k0 + kKeys > w.keys) {
                        const int v = w.slot0 + 2 * j + 1;
                        wait(full(v % G::NSLOT), (uint32_t)((v / G::NSLOT) & 1));
                        if (k0 + trow >= w.keys) {
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
                        // masked scores are overwritten in place, 32 keys at a time: rare, so short
                        // code (a prompt's chunk with a window of 1,024 takes 93 us; 16 at a time 2 %
                        // longer; masked in registers 2 %, and 5 for a long context; leaving out
                        // those 32 that every row sees 2 %)
                        if (k0 + kKeys > open_hi || k0 < open_lo) {
#pragma unroll 1
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t see = seen32(p, w.first, w.keys, pos, word, k0 + e * 32);
                                tmem_ld32(s_at + e * 32, t[0]);
                                tmem_wait_ld();
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t r[16];
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        r[k] = (see >> (16 * h + k)) & 1u ? __float_as_uint(t[0][16 * h + k]) : 0xFF800000u;
                                    tmem_st16(s_at + e * 32 + h * 16, r);
                                }
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
                        const float most = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                        const float top = c * most;
                        const bool moved = top > m + 8.f;            // also from -inf
                        if (__any_sync(0xffffffffu, moved)) {
                            const float f = moved ? ex2(m - top) : 1.f;
                            if (moved) {
                                c = c0;
                                m = c0 * most;
                                // An exponent is c s - m, rounded once, so the largest score's is what was
                                // rounded off m: up to 1/2 below 2^24, 8 below 2^28, fp32's limit at 2^32.  From
                                // 2^24 on c and m are made smaller by a power of two that leaves 2^23 of m.
                                // Scores there are apart by the rest of a unit or more, and by 2^23 times
                                // their relative difference: those that this brings nearer differ by
                                // fewer units of their last place than their sums are off by.  (With scores
                                // less the largest, times c, as two operations throughout, a prompt's chunk
                                // over 4 bits takes 4.6 % longer; by this 1.7, which are spilled registers.)
                                if (fabsf(m) >= 16777216.f) {
                                    const float less = __uint_as_float((277u << 23) - (__float_as_uint(m) & 0x7F800000u));
                                    m *= less, c *= less;
                                }
                            }
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
                        heavy = 2.f * ex2(c * most - m) >= x.x + x.y;
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
            if (c != c0)                                 // a power of two
                m *= c0 / c;
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
            const int64_t tok = w.q0 + i;
            const int head = w.head * p.group + row - i * p.group;
            float* slot = p.partial + (size_t)(2 * blockIdx.x + (w.c0 == (int)blockIdx.x)) * G::PARTIAL;
            // dual: all columns of the row; else the stream's half of them
            const int e0 = dual ? 0 : s * (D / 64), e1 = dual ? D / 32 : (s + 1) * (D / 64);
            // (the quotient is rounded to 16 bits: an approximate reciprocal, off by 2^-23, will do)
            const float f = sum == 0.f ? 0.f : __fdividef(1.f, sum);     // (NaN stays)
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
                static_cast<JoinItem*>(p.items)[w.c0] = {w.q0, w.row0, w.rows, w.head,
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

template <int DT, int D, bool KV4>
cudaError_t launch(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, int sms,
                   cudaStream_t st)
{
    auto kernel = lbv_attend_tiles_kernel<DT, D, KV4>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Geo<D, KV4>::BYTES);
    if (e != cudaSuccess)
        return e;
    const int ctas = sms < kAttendMaxCtas ? sms : kAttendMaxCtas;
    e = launch_after(kernel, dim3((unsigned)ctas), Roles<KV4>::THREADS, Geo<D, KV4>::BYTES, st, p, kmap, vmap);
    return e == cudaSuccess ? launch_attend_join(p, (lbv_dtype)DT, kRows, ctas, st) : e;
}

template <bool KV4>
cudaError_t launch_tiles(const AttendParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, lbv_dtype dt,
                         int sms, cudaStream_t st)
{
    if (dt == LBV_F16)
        return p.kv.dim == 128 ? launch<LBV_F16, 128, KV4>(p, kmap, vmap, sms, st)
                               : launch<LBV_F16, 64, KV4>(p, kmap, vmap, sms, st);
    return p.kv.dim == 128 ? launch<LBV_BF16, 128, KV4>(p, kmap, vmap, sms, st)
                           : launch<LBV_BF16, 64, KV4>(p, kmap, vmap, sms, st);
}

}  // namespace
}  // namespace lbv

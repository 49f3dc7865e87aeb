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
//     turn, by TMA; one thread issues the MMAs; commits free the slots.
//   * A row's reference maximum moves only when it grew by more than 8 (see
//     attend_rows.cu); only then are its sums in tensor memory rescaled, by the
//     row's own thread.
//   * The (item, block) pairs of the batch are divided evenly over one CTA per
//     SM, as in attend_rows.cu; a causal tile counts the blocks that it sees.
#include "attend_common.cuh"

namespace lbv {

using namespace att;

namespace {

constexpr int kKeys = 128;                       // keys per block
constexpr int kTile = 128;                       // rows per stream
constexpr int kRows = 2 * kTile;                 // rows per item
constexpr int kMinBlocks = 2;                    // least share of a CTA
constexpr int kThreads = 384;                    // copies and MMAs, then the two streams
// Registers a thread after the split: 168 * 384 at launch = 56 * 128 + 224 * 256.
constexpr int kRegsControl = 56, kRegsStream = 224;

template <int D>
struct Geo {
    static constexpr int HALF = kKeys * 128;                // 64 elements of 128 rows
    static constexpr int SLOT = (D / 64) * HALF;            // one block's K or V; one Q tile
    static constexpr int Q = 0;
    static constexpr int RING = 2 * SLOT;
    static constexpr int NSLOT = D == 128 ? 5 : 10;
    static constexpr int BARS = RING + NSLOT * SLOT;
    static constexpr int NBARS = 2 * NSLOT + 8;
    static constexpr int STATS = BARS + NBARS * 8;          // [2][128] m and sums of the streams
    static constexpr int START = STATS + 2 * kTile * 8;     // where the CTA's share begins
    static constexpr int WORDS = START + 48;                // tensor-memory address, join flag
    static constexpr int BYTES = WORDS + 16;
    static constexpr int PARTIAL = kRows * (D + 2);         // floats of one partial result
    // tensor memory columns
    static constexpr uint32_t S0 = 0, O0 = 256;             // S of stream s at S0 + 128 s
    static_assert(BYTES <= 227 * 1024, "shared memory");
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

__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
        "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n"
        ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b),
        "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// Arrives on `bar` once every MMA this thread has issued is complete.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
                 : "memory");
}

// Shared-memory matrix descriptor in 128-byte-swizzled rows: 8-row groups 1024
// bytes apart; for an operand whose rows run along the other dimension (V),
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

// ---- the CTA's share of the batch ----

// The share's first item: request, tile, head, and the item's first unit.
struct Start {
    unsigned long long total, item;
    int r, tile, head;
};

__device__ __forceinline__ int tiles_of(const AttendParams& p, const Request& q)
{
    return (int)(((int64_t)q.n * p.group + kRows - 1) / kRows);
}

// Keys and blocks of a tile of a request.
struct Tile {
    int row0, rows, i0, i1, lo, hi, block0, blocks;
};

__device__ __forceinline__ Tile tile_of(const AttendParams& p, const Request& q, int t)
{
    Tile x;
    x.row0 = t * kRows;
    x.rows = min(kRows, q.n * p.group - x.row0);
    x.i0 = x.row0 / p.group;
    x.i1 = (x.row0 + x.rows - 1) / p.group;
    key_range(p, q, x.i0, x.i1, x.lo, x.hi);
    x.block0 = x.lo / kKeys;
    x.blocks = max(1, (x.hi + kKeys - 1) / kKeys - x.block0);    // an empty row has an output too
    return x;
}

__device__ __forceinline__ unsigned long long units_of(const AttendParams& p, const Request& q)
{
    unsigned long long n = 0;
    const int tiles = tiles_of(p, q);
    for (int t = 0; t < tiles; ++t)
        n += (unsigned)tile_of(p, q, t).blocks;
    return n * (unsigned)p.kv.heads;
}

// Run by one warp: the batch's units, and where CTA c of n begins.
__device__ void find_start(const AttendParams& p, int lane, int max_ctas, int c, Start* out)
{
    unsigned long long total = 0, base = 0;
    for (int pass = 0; pass < 2; ++pass) {
        unsigned long long first = 0;
        if (pass == 1) {
            const unsigned long long want = (total + kMinBlocks - 1) / kMinBlocks;
            const unsigned n = want < (unsigned)max_ctas ? (unsigned)want : (unsigned)max_ctas;
            if ((unsigned)c >= n)
                break;
            first = (unsigned long long)c * total / n;
        }
        for (int r0 = 0; r0 < p.batch.requests; r0 += 32) {
            const int r = r0 + lane;
            unsigned long long v = 0;
            Request q;
            if (r < p.batch.requests) {
                q = request_of(p, r);
                v = units_of(p, q);
            }
            unsigned long long sum = v;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const unsigned long long o = __shfl_up_sync(0xffffffffu, sum, d);
                sum += lane >= d ? o : 0;
            }
            if (pass == 0) {
                total += __shfl_sync(0xffffffffu, sum, 31);
                continue;
            }
            const unsigned long long at = base + sum - v;
            if (v && at <= first && first < at + v) {
                unsigned long long u = at;
                int t = 0;
                Tile x = tile_of(p, q, 0);
                while (u + (unsigned long long)x.blocks * (unsigned)p.kv.heads <= first) {
                    u += (unsigned long long)x.blocks * (unsigned)p.kv.heads;
                    x = tile_of(p, q, ++t);
                }
                const int head = (int)((first - u) / (unsigned)x.blocks);
                out->r = r;
                out->tile = t;
                out->head = head;
                out->item = u + (unsigned long long)head * (unsigned)x.blocks;
            }
            base += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    if (lane == 0)
        out->total = total;
}

// A role's walk over the CTA's items.
struct Walk {
    const AttendParams& p;
    unsigned long long u, u_end, total, item;
    int ctas, r, t, tiles, head;
    bool fresh;
    Request q;
    Tile x;
    int b_first, b_last;                   // blocks of the item in this share

    __device__ Walk(const AttendParams& p_, const Start& s, int n, int c)
        : p(p_), total(s.total), item(s.item), ctas(n), r(s.r), t(s.tile), head(s.head), fresh(true)
    {
        u = first_of(c);
        u_end = first_of(c + 1);
        q = request_of(p, r);
        tiles = tiles_of(p, q);
        x = tile_of(p, q, t);
    }
    __device__ unsigned long long first_of(int c) const
    {
        return (unsigned long long)c * total / (unsigned)ctas;
    }
    __device__ int cta_of(unsigned long long v) const
    {
        return (int)(((v + 1) * (unsigned)ctas - 1) / total);
    }
    __device__ bool next()
    {
        if (u >= u_end)
            return false;
        if (!fresh) {
            item += (unsigned)x.blocks;
            if (++head == p.kv.heads) {
                head = 0;
                if (++t == tiles) {
                    t = 0;
                    do {
                        q = request_of(p, ++r);          // units remain, so a request does
                        tiles = tiles_of(p, q);
                    } while (tiles == 0 && r + 1 < p.batch.requests);
                }
                x = tile_of(p, q, t);
            }
        }
        fresh = false;
        b_first = (int)(u - item);
        const unsigned long long end = item + (unsigned)x.blocks;
        b_last = (int)((end < u_end ? end : u_end) - item);
        u = item + (unsigned)b_last;
        return true;
    }
    __device__ bool whole() const { return b_first == 0 && b_last == x.blocks; }
    __device__ bool dual() const { return x.rows > kTile; }
    __device__ int key0(int b) const { return (x.block0 + b) * kKeys; }
};

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
    Start* start = reinterpret_cast<Start*>(smem + G::START);
    uint32_t& tmem_slot = *reinterpret_cast<uint32_t*>(smem + G::WORDS);
    int& flag = *reinterpret_cast<int*>(smem + G::WORDS + 4);        // this CTA joins the parts
    auto bar = [&](int i) { return sbase + G::BARS + i * 8; };
    auto full = [&](int i) { return bar(i); };
    auto empty = [&](int i) { return bar(G::NSLOT + i); };
    const uint32_t q_full = bar(2 * G::NSLOT);                       // both Q tiles are stored
    auto s_full = [&](int s) { return bar(2 * G::NSLOT + 1 + s); };  // S of stream s is complete
    auto p_full = [&](int s) { return bar(2 * G::NSLOT + 3 + s); };  // P replaced it
    auto o_done = [&](int s) { return bar(2 * G::NSLOT + 5 + s); };  // O has the block

    if (tid == 0) {
        for (int i = 0; i < G::NSLOT; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), 1);
        }
        mbar_init(q_full, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full(s), 1);
            mbar_init(p_full(s), 4);
            mbar_init(o_done(s), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0)
        find_start(p, lane, gridDim.x, blockIdx.x, start);
    __syncthreads();
    const unsigned long long want = (start->total + kMinBlocks - 1) / kMinBlocks;
    const int ctas = (int)(want < gridDim.x ? want : gridDim.x);
    if ((int)blockIdx.x >= ctas)
        return;
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

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsControl));
        if (warp == 0) {
            // ---- copies: K and V of each block in turn ----
            Walk w(p, *start, ctas, blockIdx.x);
            const int slots = min(64, 1 << p.kv.page_shift);         // rows of a box
            const int boxes = kKeys / slots;
            int n = 0;
            while (w.next()) {
                const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
                for (int i = 2 * w.b_first; i < 2 * w.b_last; ++i) {
                    const int st = n % G::NSLOT, k0 = w.key0(i >> 1);
                    if (n >= G::NSLOT && ok)
                        ok = mbar_wait(empty(st), (uint32_t)((n / G::NSLOT - 1) & 1));
                    ++n;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok)
                        continue;
                    if (lane == 0)
                        mbar_expect_tx(full(st), G::SLOT);
                    __syncwarp();
                    for (int b = lane; b < boxes * (D / 64); b += 32) {
                        const int piece = b % boxes, half = b / boxes;
                        const int key = k0 + piece * slots;
                        int page = -1;                               // fills zeros
                        if (key < w.x.hi && key + slots > w.x.lo)
                            page = table[key >> p.kv.page_shift];
                        tma_box(sbase + G::RING + st * G::SLOT + half * G::HALF + piece * slots * 128,
                                (i & 1) ? &vmap : &kmap, half * 64,
                                key & ((1 << p.kv.page_shift) - 1), w.head, page, full(st));
                    }
                }
            }
            // the ring drains before shared memory goes away
            for (int i = 0; i < G::NSLOT; ++i)
                if (n - 1 - i >= 0 && ok)
                    ok = mbar_wait(empty((n - 1 - i) % G::NSLOT),
                                   (uint32_t)(((n - 1 - i) / G::NSLOT) & 1));
        } else if (warp == 1 && lane == 0) {
            // ---- MMAs ----
            Walk w(p, *start, ctas, blockIdx.x);
            constexpr uint32_t id_s = idesc<DT>(kKeys, false), id_o = idesc<DT>(D, true);
            auto wait = [&](uint32_t b, uint32_t parity) {
                if (ok)
                    ok = mbar_wait(b, parity);
            };
            int n = 0, items = 0;                        // slots before this item, items so far
            int np[2] = {0, 0};                          // blocks of each stream so far
            while (w.next()) {
                const int nb = w.b_last - w.b_first;
                wait(q_full, (uint32_t)(items++ & 1));
                tc_fence_after();
                auto k_slot = [&](int j) { return n + 2 * j; };
                auto v_slot = [&](int j) { return n + 2 * j + 1; };
                auto arrived = [&](int i) { wait(full(i % G::NSLOT), (uint32_t)((i / G::NSLOT) & 1)); };
                auto score = [&](int s, int tile, int j) {           // S_s = Q_tile K_j^T
                    const uint32_t a = sbase + G::Q + tile * G::SLOT;
                    const uint32_t b = sbase + G::RING + (k_slot(j) % G::NSLOT) * G::SLOT;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss(tmem + G::S0 + s * 128, desc128(a + (ks / 4) * G::HALF + (ks % 4) * 32, 0),
                               desc128(b + (ks / 4) * G::HALF + (ks % 4) * 32, 0), id_s, ks > 0);
                    commit(s_full(s));
                };
                auto value = [&](int s, int j, bool add) {           // O_s += P_s V_j
                    wait(p_full(s), (uint32_t)(np[s]++ & 1));
                    tc_fence_after();
                    const uint32_t b = sbase + G::RING + (v_slot(j) % G::NSLOT) * G::SLOT;
#pragma unroll
                    for (int ks = 0; ks < kKeys / 16; ++ks)
                        mma_ts(tmem + G::O0 + s * 128, tmem + G::S0 + s * 128 + ks * 8,
                               desc128(b + ks * 2048, G::HALF), id_o, add || ks > 0);
                    commit(o_done(s));
                };
                if (w.dual()) {
                    arrived(k_slot(0));
                    score(0, 0, 0);
                    score(1, 1, 0);
                    commit(empty(k_slot(0) % G::NSLOT));
                    for (int j = 0; j < nb; ++j) {
                        arrived(v_slot(j));
                        if (j + 1 < nb)
                            arrived(k_slot(j + 1));
                        value(0, j, j > 0);
                        if (j + 1 < nb)
                            score(0, 0, j + 1);
                        value(1, j, j > 0);
                        commit(empty(v_slot(j) % G::NSLOT));
                        if (j + 1 < nb) {
                            score(1, 1, j + 1);
                            commit(empty(k_slot(j + 1) % G::NSLOT));
                        }
                    }
                } else {
                    for (int j = 0; j < 2 && j < nb; ++j) {
                        arrived(k_slot(j));
                        score(j, 0, j);
                        commit(empty(k_slot(j) % G::NSLOT));
                    }
                    for (int j = 0; j < nb; ++j) {
                        arrived(v_slot(j));
                        value(j & 1, j, j > 1);
                        commit(empty(v_slot(j) % G::NSLOT));
                        if (j + 2 < nb) {
                            arrived(k_slot(j + 2));
                            score(j & 1, 0, j + 2);
                            commit(empty(k_slot(j + 2) % G::NSLOT));
                        }
                    }
                }
                n += 2 * nb;
            }
            // the last MMAs end before tensor memory goes away
            for (int s = 0; s < 2; ++s)
                if (np[s])
                    wait(o_done(s), (uint32_t)((np[s] - 1) & 1));
        }
        __syncwarp();
    } else {
        // ---- the streams: one row a thread ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsStream));
        Walk w(p, *start, ctas, blockIdx.x);
        const int s = (warp >> 2) - 1;                               // stream
        const int trow = tid & 127;                                  // row within the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + G::S0 + s * 128, o_at = tmem + lanes + G::O0;
        float2* stats = reinterpret_cast<float2*>(smem + G::STATS);
        // scores are c times Q's: a negative scale negates Q, a zero one clears it
        const float c = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
        const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
        int n = 0, done = 0;             // slots before this item; blocks of this stream so far
        while (w.next()) {
            const bool dual = w.dual();
            const int nb = w.b_last - w.b_first;
            // this thread's row of the item, and its Q into shared memory
            const int item_row = dual ? s * kTile + trow : trow;
            const bool in = item_row < w.x.rows;
            const int row = w.x.row0 + item_row;
            const int i = row / p.group, g = row - i * p.group;
            const int64_t tok = w.q.q0 + i;
            const int head = w.head * p.group + g;
            const int pos = in ? w.q.first + i : INT_MIN / 2;
            const uint64_t word = in && p.tree ? p.tree[tok] : 0;
            if (dual || s == 0) {
                const uint16_t* src = p.q + tok * p.q_token + (int64_t)head * p.q_head;
                unsigned char* dst = smem + G::Q + s * G::SLOT + trow * 128;
#pragma unroll
                for (int ch = 0; ch < D / 8; ++ch) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (in && p.scale_log2 != 0.f) {
                        if (p.q_wide) {
                            v = *reinterpret_cast<const uint4*>(src + ch * 8);
                        } else {
                            uint32_t e[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                e[k] = (uint32_t)src[ch * 8 + 2 * k] |
                                       ((uint32_t)src[ch * 8 + 2 * k + 1] << 16);
                            v = make_uint4(e[0], e[1], e[2], e[3]);
                        }
                        v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
                    }
                    *reinterpret_cast<uint4*>(dst + (ch >> 3) * G::HALF + (((ch & 7) ^ (trow & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(q_full);
            // keys at `open_hi` and past, or below `open_lo`, are hidden from some row of the tile
            const int r0 = w.x.row0 + (dual ? s * kTile : 0);
            const int r1 = min(r0 + kTile, w.x.row0 + w.x.rows) - 1;
            const int open_hi = p.tree ? min(w.q.keys, w.q.first)
                                       : min(w.q.keys, w.q.first + r0 / p.group + 1);
            const int open_lo = p.window > 0 ? w.q.first + r1 / p.group - p.window + 1 : 0;
            const bool idle = r0 + (warp & 3) * 32 > r1;             // no row in this warp
            float m = -INFINITY;
            float2 l = make_float2(0.f, 0.f);
            int mine = 0;                                            // blocks of this item
            for (int j = dual ? 0 : s; j < nb; j += dual ? 1 : 2, ++mine, ++done) {
                const int k0 = w.key0(w.b_first + j);
                if (ok)
                    ok = mbar_wait(s_full(s), (uint32_t)(done & 1));
                tc_fence_after();
                if (!idle) {
                    float t[4][32];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        tmem_ld32(s_at + e * 32, t[e]);
                    tmem_wait_ld();
                    if (k0 + kKeys > open_hi || k0 < open_lo) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t see = seen32(p, w.q, pos, word, k0 + e * 32);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                t[e][k] = (see >> k) & 1u ? t[e][k] : -INFINITY;
                        }
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 128; e += 2)
                        top = fmaxf(top, fmaxf(t[e >> 5][e & 31], t[e >> 5][(e & 31) + 1]));
                    top *= c;
                    const bool moved = top > m + 8.f;                // also from -inf
                    if (__any_sync(0xffffffffu, moved)) {
                        const float f = moved ? ex2(m - top) : 1.f;
                        m = moved ? top : m;
                        l.x *= f, l.y *= f;
                        if (mine > 0) {
                            if (ok)
                                ok = mbar_wait(o_done(s), (uint32_t)((done - 1) & 1));
                            tc_fence_after();
#pragma unroll 1
                            for (int e = 0; e < D / 32; ++e) {
                                float o[32];
                                tmem_ld32(o_at + s * 128 + e * 32, o);
                                tmem_wait_ld();
                                uint32_t r[32];
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    r[k] = __float_as_uint(o[k] * f);
                                tmem_st32(o_at + s * 128 + e * 32, r);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : -m;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t r[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float a = ex2(fmaf(t[2 * h + (e >> 4)][(2 * e) & 31], c, ref));
                            const float b = ex2(fmaf(t[2 * h + (e >> 4)][((2 * e) & 31) + 1], c, ref));
                            l.x += a, l.y += b;
                            r[e] = pack2<DT>(a, b);
                        }
                        tmem_st32(s_at + h * 32, r);
                    }
                    tmem_wait_st();
                }
                // slots past the context may hold anything: NaN times 0 is not 0
                if (k0 + kKeys > w.q.keys) {
                    const int v = n + 2 * j + 1;
                    if (ok)
                        ok = mbar_wait(full(v % G::NSLOT), (uint32_t)((v / G::NSLOT) & 1));
                    if (k0 + trow >= w.q.keys) {
                        unsigned char* z = smem + G::RING + (v % G::NSLOT) * G::SLOT + trow * 128;
#pragma unroll
                        for (int e = 0; e < D / 8; ++e)
                            *reinterpret_cast<uint4*>(z + (e >> 3) * G::HALF + ((e & 7) << 4)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full(s));
            }
            n += 2 * nb;

            // ---- the item's result ----
            if (mine > 0 && ok)
                ok = mbar_wait(o_done(s), (uint32_t)((done - 1) & 1));
            float sum = l.x + l.y, f0 = 1.f, f1 = 0.f;   // factors of this row in O_0 and O_1
            if (!dual) {
                stats[s * kTile + trow] = make_float2(m, sum);
                tc_fence_before();
                named_bar_sync(1, 256);
                const float2 a = stats[trow], b = stats[kTile + trow];
                m = fmaxf(a.x, b.x);
                f0 = a.x == -INFINITY ? 0.f : ex2(a.x - m);
                f1 = b.x == -INFINITY ? 0.f : ex2(b.x - m);
                sum = f0 * a.y + f1 * b.y;
            }
            tc_fence_after();
            const bool whole = w.whole();
            const int c0 = whole ? 0 : w.cta_of(w.item);
            const int c1 = whole ? 0 : w.cta_of(w.item + (unsigned)w.x.blocks - 1);
            float* slot = p.partial + (size_t)(2 * blockIdx.x + (c0 == (int)blockIdx.x)) * G::PARTIAL;
            // dual: all columns of the row; else the stream's half of them
            const int e0 = dual ? 0 : s * (D / 64), e1 = dual ? D / 32 : (s + 1) * (D / 64);
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
                    const float f = sum > 0.f ? 1.f / sum : 0.f;
                    uint32_t r[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        r[k] = sum == 0.f ? 0u : pack2<DT>(o[2 * k] * f, o[2 * k + 1] * f);
                    store_row<32>(p.out + tok * p.out_token + (int64_t)head * p.out_head + e * 32, r);
                } else if (in) {
                    float4* d = reinterpret_cast<float4*>(slot + item_row * D + e * 32);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        d[k] = sum == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                          : make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            if (in && (dual || s == 0)) {
                if (whole && p.lse) {
                    p.lse[tok * p.heads + head] = lse_of(m, sum);
                } else if (!whole) {
                    slot[kRows * D + item_row] = m;
                    slot[kRows * (D + 1) + item_row] = sum;
                }
            }
            if (!whole) {
                __threadfence();
                named_bar_sync(1, 256);
                if (tid == 128)
                    flag = atomicAdd(p.counters + c0, 1u) == (unsigned)(c1 - c0);
                named_bar_sync(1, 256);
                if (flag) {                              // every part is there: join them
                    __threadfence();
                    join_parts<DT, D, kRows>(p, w.q, w.head, w.x.row0, w.x.rows, c0, c1, tid - 128, 256);
                    if (tid == 128)
                        p.counters[c0] = 0;              // as the next call finds it
                }
            }
            // both streams are done reading O and the flag
            tc_fence_before();
            named_bar_sync(1, 256);
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
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::BYTES);
    if (e != cudaSuccess)
        return e;
    kernel<<<sms < kAttendMaxCtas ? sms : kAttendMaxCtas, kThreads, Geo<D>::BYTES, st>>>(p, kmap, vmap);
    return cudaGetLastError();
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
    return (size_t)2 * (sms < kAttendMaxCtas ? sms : kAttendMaxCtas) * kRows * (dim + 2);
}

}  // namespace lbv

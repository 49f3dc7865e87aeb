// attend4_rows.cu -- attention of few new tokens over a paged cache of 4 bits (plain
// decoding, verify calls, trees of drafted tokens).
//
// The sums of attend_rows.cu.  A quarter of the bytes leaves a quarter of the time for
// everything else, so what a key costs in instructions counts: 13 to expand 8 codes, and
// as little as can be beside them.
//   * The products are turned around: keys (then elements of a head) are the 16 rows of an
//     mma.sync tile and the queries its 8 columns,
//         S^T = K Q^T,   O^T += V^T P^T,
//     so that 8 rows (a decoded token's query heads) take half the instructions that they
//     take as rows.  Codes are expanded in the registers of the lane that holds them as an
//     operand, once for all rows of the item: which element a place of the contraction
//     stands for is free, so a lane takes a quarter of a key (in one load, with one
//     scale and bias) and, of a value, the same eighth of two keys (two permutes a word bring
//     them together).  The
//     probabilities change places by movmatrix.
//   * A team of four warps has a share of the batch.  A warp has 16 keys of every block and
//     a running maximum, sums and results of its own: the warps meet at an item's ends alone.
//   * A warp beside each team finds its items and copies blocks of 64 keys by bulk copies: a
//     chunk of a head, keys, values and scales, is one stretch of memory.  Keys are dealt to
//     a tile's rows in an order that leaves the lanes' shared-memory banks apart for keys
//     and values alike.  It hands most of its registers to the teams.
// Shares, items and references are those of attend_rows.cu, with a team in place of a CTA; the
// parts of divided items are added by a launch of their own (attend_join.cu).  (Adding them in
// this kernel, as attend_rows.cu does for small batches, cost the block's loop registers.)
//
// What bounds it (48 query over 8 key/value heads of 128): 64 requests of one token over
// 500 to 16,384 keys, 396 MB, take 93 us, 4.3 TB/s, 63 % of what a copy reaches; the 16-bit
// cache's kernel takes 215.  Issue slots are 69 % busy with 71 million instructions, half of them
// codes', and their pipes near half; the copies alone (no codes expanded) take 67 us.
// (Three teams an SM in place of four: 2 % longer.)  More rows cost their products and probabilities: 32 requests over 7,000
// keys take 68 us with 6 rows each, 87 with 12, 120 with 24.  A single request is its launches, its
// start and its join: one token over 2,011 keys 9.5 us.
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

// Keys per block, 16 a warp.  (128, 32 a warp, save what a block costs beside its keys, and divide
// small batches less evenly: in an earlier version of this kernel 64 requests of one token took 6 %
// less, a window of 2,048 over 32 requests 14 % more, four tokens after 200,000 16 % more.)
constexpr int kBlock = 64;
constexpr int kMinUnits = 2;                     // the least share of a team
constexpr int kKeyWarps = 4, kTeam = kKeyWarps * 32;
// A reference that every score passes, negated: nothing has been seen yet.
constexpr float kNone = 3.402823466e38f;
// References from here on are worth a product that is rounded before they are taken from it: in a
// fused multiply-add the largest score's exponent is what was rounded off the reference, up to
// half a unit of its last place.  Below 2^12 that is 2^-13 or less, and 2^x rounds to 1 in 16 bits;
// it is up to 1 below 2^25, 8 below 2^28 and more than fp32's exponents from 2^32 on.
constexpr float kLarge = 4096.f;
constexpr int kItems = 16;                        // items that a team's warps may be apart: stages, and one

// What a team needs to know of an item.
struct alignas(16) Item {
    int q0, first, keys;   // of its request
    int row0, rows, head;
    int key0, nb;          // its first key and its blocks in this share; 0 blocks: no more items
    int skip, jump;        // keys left out before block `jump` (behind the sinks)
    int c0, c1;            // shares that hold a part of it
};
static_assert(sizeof(Item) == 48, "ring entry");

// NT: tiles of 8 rows of an item.
template <int D, int NT>
struct Geo {
    static constexpr int ROWS = 8 * NT;
    // (32 trees: 3 in place of 6 160 us, these 151, 10 156)
    static constexpr int EXTRA = NT == 1 ? 3 : 6;           // units of an item beside its blocks
    // teams on an SM, and registers a thread after the split: 96 * 640 at launch = 104 * 512 +
    // 64 * 128, 128 * 512 = 152 * 384 + 56 * 128
    static constexpr int TEAMS = NT == 1 ? 4 : 3;
    static constexpr int REGS = NT == 1 ? 104 : 152, HELPER = NT == 1 ? 64 : 56;
    static constexpr int THREADS = TEAMS * kTeam + 128;
    static constexpr int STAGE = kBlock * 72 * (D / 64);
    // (two stages, and four, take 1 to 4 % longer)
    static constexpr int NST = D == 64 ? 6 : 3;
    static constexpr int SLOT = ROWS * (D + 3);             // floats of one partial result
    // a team's shared memory: the ring, the warps' results, the queries as the lanes want them (in
    // registers: one tile's cost 1 %, two tiles' 6 %, by what they leave to the rest)
    static constexpr int JOIN = NST * STAGE;
    static constexpr int JROWS = 8;                       // rows joined at a time
    static constexpr int QUERIES = JOIN + kKeyWarps * JROWS * D * 4;
    static constexpr int STATS = QUERIES + NT * 32 * (D / 8) * 4;   // [4][ROWS] maxima, sums
    static constexpr int WORDS = STATS + 2 * kKeyWarps * ROWS * 4;  // uint64 [ROWS]: the rows' words of the tree
    static constexpr int ITEMS = WORDS + 8 * ROWS;
    static constexpr int START = ITEMS;                     // where the share begins, before its first item
    static constexpr int BARS = ITEMS + kItems * 48;        // full, empty, items
    static constexpr int THERE = BARS + (2 * NST + kItems) * 8;     // a block's chunks that exist
    static constexpr int SIZE = (THERE + NST * 4 + 127) / 128 * 128;
    static constexpr int BYTES = TEAMS * SIZE;
    static_assert(ITEMS % 16 == 0 && BARS % 8 == 0 && sizeof(Start) <= kItems * 48 && NST + 1 < kItems && WORDS % 8 == 0, "layout");
    static_assert(BYTES <= 227 * 1024, "room");
};

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

// The 8 x 8 matrix of 16-bit values that the warp holds, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

// Whether any of the team's threads says so; all of them meet here.
__device__ __forceinline__ bool any_of_team(int bar, bool mine)
{
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %2, 0;\n bar.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(any)
        : "r"(bar), "r"((uint32_t)mine)
        : "memory");
    return any != 0;
}

template <int DT, int D, int NT>
__global__ void __launch_bounds__(Geo<D, NT>::THREADS, 1)
    lbv_attend4_rows_kernel(const __grid_constant__ AttendParams p)
{
    using G = Geo<D, NT>;
    constexpr int ROWS = G::ROWS, PARTS = D / 64;
    using S = Shape<ROWS, kBlock, G::EXTRA>;
    extern __shared__ __align__(1024) unsigned char smem_all[];
    const int tid = threadIdx.x, lane = tid & 31;
    const bool helper = tid >= G::TEAMS * kTeam;             // (its last warps may have no team)
    const int team = helper ? (tid - G::TEAMS * kTeam) >> 5 : tid / kTeam, warp = (tid >> 5) & 3;
    unsigned char* smem = smem_all + team * G::SIZE;
    const uint32_t sbase = smem_u32(smem);
    const int share = team * gridDim.x + blockIdx.x;         // the SMs first, then their teams
    auto full = [&](unsigned st) { return sbase + G::BARS + st * 8; };
    auto empty = [&](unsigned st) { return sbase + G::BARS + (G::NST + st) * 8; };
    auto item_full = [&](unsigned i) { return sbase + G::BARS + (2 * G::NST + i % kItems) * 8; };
    Item* items = reinterpret_cast<Item*>(smem + G::ITEMS);

    if (tid % kTeam == 0 && !helper) {
        for (int i = 0; i < G::NST; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kKeyWarps);
        }
        for (int i = 0; i < kItems; ++i)
            mbar_init(item_full(i), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    __syncthreads();
    after_previous();
    bool ok = true;
    const int cs = kv4::chunk_shift(p.kv), chunk_bytes = kv4::slot_bytes(D) << cs;

    if (helper) {
        // ---- the share's items, and copies: a lane has a chunk of a block ----
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(G::HELPER));
        if (team >= G::TEAMS)
            return;
        if (lane == 0)
            static_cast<JoinItem*>(p.items)[share].rows = 0;
        Start* start = reinterpret_cast<Start*>(smem + G::START);
        find_start<S>(p, lane, gridDim.x * G::TEAMS, kMinUnits, share, start);
        __syncwarp();
        const Start begin = *start;
        __syncwarp();                                        // the items take its place
        const int64_t page_bytes = kv4::page_bytes(p.kv);
        unsigned it = 0, n = 0;                              // items published, blocks asked for
        auto publish = [&](const Item& x) {
            if (lane == 0) {
                items[it % kItems] = x;
                mbar_arrive(item_full(it));                  // releases the stores
            }
            ++it;
        };
        if (share < begin.ctas) {
            Walk<S> w(p, begin, share);
            while (ok && w.next()) {
                const int* table = p.batch.block_table + (int64_t)w.r * p.batch.table_stride;
                const uint8_t* base = kv4::chunk(p.kv, 0, w.head, 0);
                auto page_of = [&](int b) {                  // of the lane's chunk, -1: zeros
                    const int key = w.key0(b) + (lane << cs);
                    return b < w.b_last && lane << cs < kBlock && wanted(p, w.x.lo, w.x.hi, key, 1 << cs)
                               ? table[key >> p.kv.page_shift]
                               : -1;
                };
                int next = page_of(w.b_first);
#pragma unroll 1
                for (int b = w.b_first; b < w.b_last; ++b) {
                    const unsigned st = n % G::NST;
                    const int page = next;
                    next = page_of(b + 1);
                    // A stage is asked for again when it has been read, and its last copies have
                    // landed (readers that gave up free it all the same).
                    if (n >= G::NST) {
                        const uint32_t parity = (n / G::NST - 1) & 1;
                        ok = mbar_wait(empty(st), parity, p.wait_limit) &&
                             mbar_wait(full(st), parity, p.wait_limit);
                    }
                    ok = __all_sync(0xffffffffu, ok && (n < p.first_copies || share > 0));
                    if (!ok)                                 // no more copies, and no more items: places
                        break;                               // of those that are known may still be read
                    if (b == w.b_first) {
                        const bool whole = w.whole(), split = b < w.x.near;      // sinks, then a window
                        publish({w.q.q0, w.q.first, w.q.keys, w.x.row0, w.x.rows, w.head, w.key0(b),
                                 w.b_last - b, w.x.gap * kBlock, split ? w.x.near - b : -1,
                                 whole ? 0 : w.first_cta(), whole ? 0 : w.last_cta()});
                    }
                    ++n;
                    const bool go = page >= 0 && page < p.kv.pages;
                    const unsigned there = __ballot_sync(0xffffffffu, go);
                    if (lane == 0) {
                        // all ones: every key of the block exists
                        const int chunks = __popc(there);
                        reinterpret_cast<uint32_t*>(smem + G::THERE)[st] =
                            chunks == kBlock >> cs && w.key0(b) + kBlock <= w.q.keys ? ~0u : there;
                        mbar_expect_tx(full(st), chunks * chunk_bytes);
                    }
                    __syncwarp();
                    if (go) {
                        const int s = (w.key0(b) + (lane << cs)) & ((1 << p.kv.page_shift) - 1);
                        bulk_copy(sbase + st * G::STAGE + lane * chunk_bytes,
                                  base + page * page_bytes + (s >> cs) * chunk_bytes, chunk_bytes, full(st));
                    }
                }
            }
        }
        if (ok)
            publish(Item{});
        // the copies land before shared memory goes away, also after a wait that ran out
        for (unsigned i = 1; i <= G::NST && i <= n; ++i)
            if (!mbar_wait(full((n - i) % G::NST), ((n - i) / G::NST) & 1, p.wait_limit))
                ok = false;
        if (!ok && lane == 0)
            atomicOr(p.status, 1u);
        return;
    }

    // ---- the keys ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(G::REGS));
    const int g = lane >> 2, t = lane & 3, bar = 1 + team;
    // Row g of a tile is key g, or its neighbour for g >= 4, of this warp's 16 (and row g + 8 the
    // eighth after it): the keys of a quad's lanes, and of its 2 t-th and 2 t + 1-th rows, then
    // lie in four different rows of 32 bytes modulo 128.
    auto key_at = [](int r) { return r ^ ((r >> 2) & 1); };
    auto codes_of = [&](int key) { return (key >> cs) * chunk_bytes + (key & ((1 << cs) - 1)) * 32; };
    auto pair_of = [&](int key) { return (key >> cs) * chunk_bytes + (D << cs) + (key & ((1 << cs) - 1)) * 4; };
    const int k_key = warp * 16 + key_at(g), v_key0 = warp * 16 + key_at(2 * t), v_key1 = warp * 16 + key_at(2 * t + 1);
    // eight keys on: codes, pairs
    const uint32_t far = (uint32_t)chunk_bytes;
    const uint32_t eight = cs == 3 ? far : 256u, eight4 = cs == 3 ? far : 32u;
    // a quarter of a key, a lane's own t-th; an eighth of two values, its g-th: the plane of 64
    // elements it is in, and the bytes in a row of it
    const uint32_t k_part = D == 128 ? t >> 1 : 0, v_part = PARTS + (D == 128 ? g >> 2 : 0);
    const uint32_t k_at = sbase + codes_of(k_key) + (k_part * 32 << cs) + (D == 128 ? (t & 1) * 16 : t * 8),
                   k_pair = sbase + pair_of(k_key) + (k_part * 4 << cs);
    const uint32_t v_bytes = (v_part * 32 << cs) + (D == 128 ? (g & 3) * 8 : g * 4);
    const uint32_t v_at0 = sbase + codes_of(v_key0) + v_bytes, v_at1 = sbase + codes_of(v_key1) + v_bytes;
    // The two values' pairs are neighbours, for t >= 2 the other way round: what to take of them.
    const uint32_t v_pair = sbase + pair_of(warp * 16 + 2 * t) + (v_part * 4 << cs);
    const uint32_t take_scales = t < 2 ? 0x5410 : 0x1054, take_biases = t < 2 ? 0x7632 : 0x3276;
    const kv4::Constants constants = kv4::constants<DT>();
    // scores are c times the products; a scale of zero clears Q
    const float c = p.scale_log2 == 0.f ? 1.f : p.scale_log2;
    const float hidden = c < 0.f ? INFINITY : -INFINITY;
    const uint32_t queries = sbase + G::QUERIES;
    float* joint = reinterpret_cast<float*>(smem + G::JOIN);
    float* stats = reinterpret_cast<float*>(smem + G::STATS);
    uint64_t* words = reinterpret_cast<uint64_t*>(smem + G::WORDS);
    unsigned n = 0;
    for (unsigned it = 0;; ++it) {
        // one warp waits for the item, and all of them hear whether it came
        bool stop = false;
        if (warp == 0) {
            if (ok)
                ok = mbar_wait(item_full(it), (it / kItems) & 1, p.wait_limit);
            stop = !ok || items[it % kItems].nb == 0;
        }
        if (any_of_team(bar, stop))
            break;
        const Item& w = items[it % kItems];
        const int nb = w.nb, item_rows = w.rows;
        // The queries as the second operand: lane (g, t) has the t-th quarter of row g, a pair of
        // elements a word.  (Every warp writes all of them: the values are alike.)
        constexpr int QR = D / 8;                                // words of a row of a tile
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int row = w.row0 + 8 * i + g;
            const bool in = 8 * i + g < item_rows && p.scale_log2 != 0.f;
            const int tok = token_of(p, row);
            const uint16_t* src = p.q + (int64_t)(w.q0 + (in ? tok : 0)) * p.q_token +
                                  (int64_t)(w.head * p.group + (in ? row - tok * p.group : 0)) * p.q_head + t * (D / 4);
            uint32_t q[QR];
            if (!in) {
#pragma unroll
                for (int e = 0; e < QR; ++e)
                    q[e] = 0;
            } else if (p.q_wide) {
#pragma unroll
                for (int h = 0; h < QR / 4; ++h) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + h * 8);
                    q[4 * h] = v.x, q[4 * h + 1] = v.y, q[4 * h + 2] = v.z, q[4 * h + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < QR; ++e)
                    q[e] = (uint32_t)src[2 * e] | ((uint32_t)src[2 * e + 1] << 16);
            }
#pragma unroll
            for (int e = 0; e < QR / 4; ++e)
                *reinterpret_cast<uint4*>(smem + G::QUERIES + ((i * (QR / 4) + e) * 32 + lane) * 16) =
                    make_uint4(q[4 * e], q[4 * e + 1], q[4 * e + 2], q[4 * e + 3]);
        }
        if (p.tree && tid % kTeam < item_rows)
            words[tid % kTeam] = p.tree[w.q0 + token_of(p, w.row0 + tid % kTeam)];
        named_bar_sync(bar, kTeam);
        float o[NT][D / 16][4];                                  // tile j: elements g D / 8 + 2 j, and the next
        float2 minus[NT], l[NT];                                 // references, negated, and sums of rows 2 t and 2 t + 1
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            minus[i] = make_float2(kNone, kNone);
            l[i] = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
        }
        // keys below `open_lo` or at `open_hi` and past are hidden from some row
        const int open_hi = p.tree ? min(w.keys, w.first)
                                   : min(w.keys, w.first + token_of(p, w.row0) + 1);
        const int open_lo =
            p.window > 0 ? w.first + token_of(p, w.row0 + item_rows - 1) - p.window + 1 : 0;

        bool far = false;                                        // a reference of the warp passes kLarge
        int k0 = w.key0 - kBlock;
        const int jump = w.jump;
#pragma unroll 1
        for (int j = 0; j < nb; ++j, ++n) {
            const unsigned st = n % G::NST;
            k0 += kBlock;
            if (j == jump)
                k0 += w.skip;
            if (!mbar_try(full(st), (n / G::NST) & 1) && ok)
                ok = mbar_wait(full(st), (n / G::NST) & 1, p.wait_limit);
            const uint32_t there = load4(sbase + G::THERE + st * 4);
            // whether a key of the block exists: slots past the context hold anything
            auto exists = [&](int key) { return ((there >> (key >> cs)) & 1) && k0 + key < w.keys; };
            const uint32_t stage = st * G::STAGE;
            // ---- scores of 16 keys ----
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
            {
                constexpr int W = D / 32;                        // words of 8 elements
                uint32_t v[2][W], sc[2], bi[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {                    // rows g and g + 8
                    if constexpr (W == 4) {
                        load16(k_at + stage + h * eight, v[h]);
                    } else {
                        const uint2 x = load8(k_at + stage + h * eight);
                        v[h][0] = x.x, v[h][1] = x.y;
                    }
                    sc[h] = load4(k_pair + stage + h * eight4);
                }
                if (there != ~0u) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        sc[h] = exists(k_key + 8 * h) ? sc[h] : 0u;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    bi[h] = kv4::both_biases(sc[h]);
                    sc[h] = kv4::both_scales(sc[h]);
                }
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    uint32_t e[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        kv4::expand<DT>(v[h][u], sc[h], bi[h], constants, e[h]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {                // 4 of them a step
                        const uint32_t a[4] = {e[0][2 * k], e[1][2 * k], e[0][2 * k + 1], e[1][2 * k + 1]};
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint2 q = load8(queries + ((i * (QR / 4) + u) * 32 + lane) * 16 + k * 8);
                            mma<DT>(s[i], a, q.x, q.y);
                        }
                    }
                }
            }
            // ---- their probabilities ----
            const int key0 = k0 + warp * 16;
            if (key0 + 16 > open_hi || key0 < open_lo) {         // rare, so short code
                const int mine = key_at(g);
#pragma unroll 1
                for (int r = 0; r < ROWS; r += 8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {                // rows r + 2 t and the next
                        const int row = r + 2 * t + h;
                        uint32_t see = 0;
                        if (row < item_rows)
                            see = seen32(p, w.first, w.keys, w.first + token_of(p, w.row0 + row),
                                         p.tree ? words[row] : 0, key0) >> mine;
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            if (8 * i == r) {
                                s[i][h] = see & 1 ? s[i][h] : hidden;
                                s[i][2 + h] = (see >> 8) & 1 ? s[i][2 + h] : hidden;
                            }
                    }
                }
            }
            // Exponents, for the references as they are: c s less the reference, rounded once.  From
            // references of kLarge on (`far`, until the item's end) every block comes to what
            // follows, and the product is rounded first.  (64 requests of one token take 0.9 % longer by
            // the flag, 1.3 with the product rounded throughout; four tokens after 200,000, 1.5 and 2.)
            float2 x[NT][2];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[i][h] = fma2(make_float2(s[i][2 * h], s[i][2 * h + 1]), make_float2(c, c), minus[i]);
                    top = fmaxf(top, fmaxf(x[i][h].x, x[i][h].y));
                }
            if (__any_sync(0xffffffffu, far || top > 8.f)) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float& from = h ? minus[i].y : minus[i].x;
                        float top = fmaxf(c * s[i][h], c * s[i][2 + h]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        if (top + from > 8.f) {
                            const float f = ex2(-from - top);
                            from = -top;
                            far = far || fabsf(top) >= kLarge;
                            (h ? l[i].y : l[i].x) *= f;
#pragma unroll
                            for (int j = 0; j < D / 16; ++j)
                                o[i][j][h] *= f, o[i][j][2 + h] *= f;
                        }
                    }
                far = __any_sync(0xffffffffu, far);
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // (packed, mul.rn and add.rn became one fma all the same)
                        const float a = s[i][2 * h], b = s[i][2 * h + 1];
                        x[i][h] = far ? add2(make_float2(__fmul_rn(c, a), __fmul_rn(c, b)), minus[i])
                                      : fma2(make_float2(a, b), make_float2(c, c), minus[i]);
                    }
            }
            uint32_t pf[NT][2];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 y = make_float2(ex2(x[i][h].x), ex2(x[i][h].y));
                    l[i] = add2(l[i], y);
                    pf[i][h] = transposed(pack2<DT>(y.x, y.y));
                }
            // ---- and their values ----
            {
                constexpr int W = D / 64;                        // words of 8 elements
                uint32_t v[2][2][W], sc[2], bi[2];               // of two pairs of keys
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (W == 2) {
                        const uint2 a = load8(v_at0 + stage + h * eight), b = load8(v_at1 + stage + h * eight);
                        v[h][0][0] = a.x, v[h][0][1] = a.y, v[h][1][0] = b.x, v[h][1][1] = b.y;
                    } else {
                        v[h][0][0] = load4(v_at0 + stage + h * eight), v[h][1][0] = load4(v_at1 + stage + h * eight);
                    }
                    uint2 f = load8(v_pair + stage + h * eight4);
                    if (there != ~0u) {
                        const int key = warp * 16 + 8 * h + 2 * t;
                        f.x = exists(key) ? f.x : 0u;
                        f.y = exists(key + 1) ? f.y : 0u;
                    }
                    sc[h] = __byte_perm(f.x, f.y, take_scales), bi[h] = __byte_perm(f.x, f.y, take_biases);
                }
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    uint32_t e[2][2][4];                         // even and odd elements
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        kv4::expand<DT>(__byte_perm(v[h][0][u], v[h][1][u], 0x5410), sc[h], bi[h], constants, e[h][0]);
                        kv4::expand<DT>(__byte_perm(v[h][0][u], v[h][1][u], 0x7632), sc[h], bi[h], constants, e[h][1]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t a[4] = {e[0][0][j], e[0][1][j], e[1][0][j], e[1][1][j]};
#pragma unroll
                        for (int i = 0; i < NT; ++i)
                            mma<DT>(o[i][u * 4 + j], a, pf[i][0], pf[i][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(st));
        }

        // ---- the item's result: the warps' sums are joined ----
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = h ? l[i].y : l[i].x;
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (g == 0) {
                    stats[warp * ROWS + 8 * i + 2 * t + h] = h ? -minus[i].y : -minus[i].x;
                    stats[(kKeyWarps + warp) * ROWS + 8 * i + 2 * t + h] = sum;
                }
            }
        named_bar_sync(bar, kTeam);
        const int c0 = w.c0, c1 = w.c1;
        const bool whole = c0 == c1;
        Request q;
        q.q0 = w.q0;
        float* slot = p.partial + (size_t)(2 * share + (c0 == share)) * G::SLOT;
        auto top_of = [&](int r) {
            const float* q = stats + r;
            return fmaxf(fmaxf(q[0], q[ROWS]), fmaxf(q[2 * ROWS], q[3 * ROWS]));
        };
#pragma unroll
        for (int r0 = 0; r0 < ROWS; r0 += G::JROWS) {
            if (r0 >= item_rows)
                break;
            if (r0 > 0)
                named_bar_sync(bar, kTeam);                         // the rows before have been added
#pragma unroll
            for (int i = 0; i < G::JROWS / 8; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tile = r0 / 8 + i, r = 8 * tile + 2 * t + h;
                    const float f = ex2((h ? -minus[tile].y : -minus[tile].x) - top_of(r));
                    float* d = joint + (warp * G::JROWS + 8 * i + 2 * t + h) * D + g * (D / 8);
#pragma unroll
                    for (int j = 0; j < D / 16; j += 2)
                        *reinterpret_cast<float4*>(d + 2 * j) = make_float4(f * o[tile][j][h], f * o[tile][j][2 + h],
                                                                            f * o[tile][j + 1][h], f * o[tile][j + 1][2 + h]);
                }
            named_bar_sync(bar, kTeam);
            const int rows = min(G::JROWS, item_rows - r0);
            for (int i = tid % kTeam; i < rows * (D / 4); i += kTeam) {
                const int r = i / (D / 4), d4 = i % (D / 4);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                float total = 0.f;
                const float top = top_of(r0 + r);
#pragma unroll
                for (int k = 0; k < kKeyWarps; ++k) {
                    const float4 a = *reinterpret_cast<const float4*>(joint + (k * G::JROWS + r) * D + 4 * d4);
                    sum.x += a.x, sum.y += a.y, sum.z += a.z, sum.w += a.w;
                    total += ex2(stats[k * ROWS + r0 + r] - top) * stats[(kKeyWarps + k) * ROWS + r0 + r];
                }
                if (whole) {
                    finish4<DT>(p, q, w.head, w.row0 + r0 + r, d4, sum, top, total, total);
                } else {
                    *reinterpret_cast<float4*>(slot + (r0 + r) * D + 4 * d4) = sum;
                    if (d4 == 0) {
                        slot[ROWS * D + r0 + r] = top;
                        slot[ROWS * (D + 1) + r0 + r] = slot[ROWS * (D + 2) + r0 + r] = total;
                    }
                }
            }
        }
        if (!whole && tid % kTeam == 0 && c0 == share)
            static_cast<JoinItem*>(p.items)[c0] = {w.q0, w.row0, item_rows, w.head, c1 - c0 + 1};
        named_bar_sync(bar, kTeam);                                 // statistics and results have been read
    }
    if (!ok && lane == 0)
        atomicOr(p.status, 1u);
}

template <int DT, int D, int NT>
cudaError_t launch(const AttendParams& p, int sms, cudaStream_t st)
{
    using G = Geo<D, NT>;
    auto kernel = lbv_attend4_rows_kernel<DT, D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::BYTES);
    if (e != cudaSuccess)
        return e;
    const int ctas = std::min(sms, kAttendMaxCtas / G::TEAMS);
    e = launch_after(kernel, dim3((unsigned)ctas), G::THREADS, G::BYTES, st, p);
    return e == cudaSuccess ? launch_attend_join(p, (lbv_dtype)DT, G::ROWS, ctas * G::TEAMS, st) : e;
}

template <int DT, int D>
cudaError_t launch_rows(const AttendParams& p, int sms, cudaStream_t st)
{
    const int64_t rows = attend_average_rows(p);
    return rows <= 8 ? launch<DT, D, 1>(p, sms, st) : rows <= 16 ? launch<DT, D, 2>(p, sms, st) : launch<DT, D, 3>(p, sms, st);
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
    // two slots a team: three teams an SM with 24 rows, more than four with 8
    return (size_t)2 * 3 * std::min(sms, kAttendMaxCtas / 3) * 24 * (dim + 3);
}

}  // namespace lbv

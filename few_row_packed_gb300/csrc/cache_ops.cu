// cache_ops.cu -- what a program does to a paged cache between steps: reading tokens
// back, closing up the accepted ones of a tree, copying pages.  All three move bytes and
// are bound by memory, or with few bytes by a launch and round trips to memory:
// 8191 tokens of 8 heads of 128 read from 4 bits take 9.2 us (43 MB, 4.6 TB/s; one token a block
// 14.5), the accepted ones of 64 requests' trees 3.2 us (four round trips: counts, page, tokens,
// stores; 4.4 from Python), 256 pages of 262,144 bytes 22 us (134 MB, 6.1 TB/s, 90 % of what a copy
// reaches).
#include "kv4.cuh"
#include "rope_rows.cuh"

namespace lbv {

using namespace rope;

namespace {

constexpr int kThreads = 256;

// ---- tokens as rows ----
//
// A thread takes 8 elements of a head's key or value, a block kTokens tokens: what a
// token's place takes is four loads that wait for one another, so many are under way.

constexpr int kTokens = 4;

template <int DT, bool PACKED>
__global__ void __launch_bounds__(kThreads) lbv_kv_read_kernel(const __grid_constant__ ReadParams p)
{
    __shared__ int where[kTokens][2];              // request, then page (-1: reads as zeros, -2: no request); slot
    const int tok0 = blockIdx.x * kTokens, tid = threadIdx.x;
    after_previous();
    if (tid < kTokens)
        where[tid][0] = -1;
    __syncthreads();
    for (int r = tid; r < p.batch.requests; r += kThreads) {
        const int lo = p.batch.q_start[r], hi = p.batch.q_start[r + 1];
        for (int tok = max(lo, tok0); tok < min(min(hi, p.batch.tokens), tok0 + kTokens); ++tok) {
            where[tok - tok0][0] = r;
            where[tok - tok0][1] = p.batch.kv_len[r] - hi + tok;
        }
    }
    __syncthreads();
    if (tid < kTokens) {
        const int req = where[tid][0], pos = where[tid][1];
        where[tid][0] = req < 0 ? -2 : page_of(p.batch, p.kv, req, pos);
        where[tid][1] = pos & ((1 << p.kv.page_shift) - 1);
    }
    __syncthreads();
    const int shift = p.kv.dim == 128 ? 4 : 3, per = p.kv.heads << shift;
    const int units = 2 * per, step = kThreads * gridDim.y;
    for (int it = blockIdx.y * kThreads + tid; it < units; it += step) {
        const int which = it >= per, e = it - which * per, head = e >> shift, at = (e - (head << shift)) * 8;
        if (!p.out[which])
            continue;
        uint4 v[kTokens];
        uint32_t pair[kTokens], word[kTokens];
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {        // all of them in flight
            const int page = where[i][0], slot = where[i][1];
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            pair[i] = word[i] = 0;
            if (page < 0)
                continue;
            if constexpr (PACKED) {
                const int cs = kv4::chunk_shift(p.kv), s = slot & ((1 << cs) - 1), planes = p.kv.dim >> 5;
                const int plane = which * (planes >> 1) + (at >> 6);
                const uint8_t* c = kv4::chunk(p.kv, page, head, slot);
                pair[i] = *reinterpret_cast<const uint32_t*>(c + kv4::scale_at(planes, plane, s, cs));
                word[i] = *reinterpret_cast<const uint32_t*>(c + kv4::codes_at(plane, s, cs) + ((at >> 3) & 7) * 4);
            } else {
                v[i] = *reinterpret_cast<const uint4*>((which ? p.kv.v : p.kv.k) + page * p.kv.page_stride +
                                                       slot * p.kv.token_stride + head * p.kv.head_stride + at);
            }
        }
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if (where[i][0] == -2)
                continue;                          // a row of no request
            if constexpr (PACKED) {
                uint32_t x[4];
                kv4::expand<DT>(word[i], kv4::both_scales(pair[i]), kv4::both_biases(pair[i]), kv4::constants<DT>(), x);
                v[i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            uint16_t* d = p.out[which] + (tok0 + i) * p.out_token[which] + head * p.out_head[which] + at;
            if (p.wide) {
                *reinterpret_cast<uint4*>(d) = v[i];
            } else {
                const uint32_t r[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    d[j] = (uint16_t)(r[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

// ---- tokens that stay ----
//
// One block takes a request's new tokens in one head.  A token's place may be another's
// source, so the block loads all of them before it stores the first: 64 tokens of 128
// 16-bit elements, keys and values, are 2048 vectors of 16 bytes, eight a thread.

constexpr int kMost = 64;                          // new tokens that a word names

struct Move {
    int64_t from, to;                              // elements, or bytes of the chunks if packed; from -1: none
    int s0, s1;                                    // slots of the chunks
};

template <bool PACKED>
__global__ void __launch_bounds__(kThreads)
    lbv_kv_keep_kernel(const __grid_constant__ lbv_batch b, const __grid_constant__ KvView kv, const uint64_t* kept,
                       int32_t* left)
{
    __shared__ Move moves[kMost];
    const int r = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
    after_previous();
    const int n = b.q_start[r + 1] - b.q_start[r], first = b.kv_len[r] - n;
    uint64_t word = n > 0 ? kept[r] : 0;
    if (n > 0 && n < kMost)
        word &= (1ull << n) - 1;
    const bool all = word == ~0ull;                // also of more than a word names
    const int count = __popcll(word);
    if (left && head == 0 && tid == 0)
        left[r] = first + (all ? n : count);
    const int still = all ? kMost : __ffsll((long long)~word) - 1;    // the first of them stay where they are
    const int moving = count - still;
    if (moving <= 0)
        return;
    const int cs = PACKED ? kv4::chunk_shift(kv) : 0;
    if (tid >= still && tid < kMost && (word >> tid) & 1) {
        const int to = __popcll(word & ((1ull << tid) - 1));
        const int page0 = page_of(b, kv, r, first + tid), page1 = page_of(b, kv, r, first + to);
        const int mask = (1 << kv.page_shift) - 1, s0 = (first + tid) & mask, s1 = (first + to) & mask;
        Move m = {-1, -1, 0, 0};
        if (page0 >= 0 && page1 >= 0) {
            if constexpr (PACKED)
                m = {kv4::chunk(kv, page0, head, s0) - kv.packed, kv4::chunk(kv, page1, head, s1) - kv.packed,
                     s0 & ((1 << cs) - 1), s1 & ((1 << cs) - 1)};
            else
                m = {page0 * kv.page_stride + s0 * kv.token_stride + head * kv.head_stride,
                     page1 * kv.page_stride + s1 * kv.token_stride + head * kv.head_stride, 0, 0};
        }
        moves[to - still] = m;
    }
    __syncthreads();
    if constexpr (PACKED) {
        // `planes` rows of 32 bytes of codes a token, and as many pairs of scale and bias
        const int planes = kv.dim >> 5, row = tid / planes, plane = tid - row * planes;
        uint4 v[2];
        uint32_t pair = 0;
        const Move m = row < moving ? moves[row] : Move{-1, -1, 0, 0};
        if (m.from >= 0) {
            const uint4* src = reinterpret_cast<const uint4*>(kv.packed + m.from + kv4::codes_at(plane, m.s0, cs));
            v[0] = src[0], v[1] = src[1];
            pair = *reinterpret_cast<const uint32_t*>(kv.packed + m.from + kv4::scale_at(planes, plane, m.s0, cs));
        }
        __syncthreads();
        if (m.from >= 0) {
            uint4* d = reinterpret_cast<uint4*>(kv.packed + m.to + kv4::codes_at(plane, m.s1, cs));
            d[0] = v[0], d[1] = v[1];
            *reinterpret_cast<uint32_t*>(kv.packed + m.to + kv4::scale_at(planes, plane, m.s1, cs)) = pair;
        }
    } else {
        const int shift = kv.dim == 128 ? 4 : 3;               // vectors of a key
        const int all = moving << (shift + 1);
        constexpr int U = kMost * 32 / kThreads;
        uint4 v[U];
        auto at = [&](int i, bool to) {
            const Move& m = moves[i >> (shift + 1)];
            uint16_t* base = (i >> shift) & 1 ? kv.v : kv.k;
            return reinterpret_cast<uint4*>(base + (to ? m.to : m.from) + (i & ((1 << shift) - 1)) * 8);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + u * kThreads;
            if (i < all && moves[i >> (shift + 1)].from >= 0)
                v[u] = *at(i, false);
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + u * kThreads;
            if (i < all && moves[i >> (shift + 1)].from >= 0)
                *at(i, true) = v[u];
        }
    }
}
static_assert(kMost * 4 <= kThreads, "a thread takes one row of codes");

// ---- pages ----
//
// A block copies a part of a page: kAhead vectors of 16 bytes a thread in flight.

constexpr int kAhead = 8;

struct CopyParams {
    KvView kv;
    const int32_t* src;
    const int32_t* dst;
    int vectors, parts;                            // of a page, keys and values; blocks that copy one
    int inner;                                     // rows of the dimension with the smaller stride
    int shift;                                     // log2 of the vectors of a row
    int64_t inner_stride, outer_stride;
};

template <bool PACKED>
__global__ void __launch_bounds__(kThreads) lbv_kv_copy_kernel(const __grid_constant__ CopyParams p)
{
    after_previous();
    const int pair = blockIdx.x / p.parts, part = blockIdx.x - pair * p.parts;
    const int from = p.src[pair], to = p.dst[pair];
    if (from < 0 || from >= p.kv.pages || to < 0 || to >= p.kv.pages || from == to)
        return;
    const int64_t page = PACKED ? kv4::page_bytes(p.kv) : 0;
    const int half = PACKED ? 0 : p.vectors / 2;
    auto offset = [&](int i) {                     // of vector i of the keys (or values) in a page
        const int row = i >> p.shift, o = row / p.inner;
        return o * p.outer_stride + (row - o * p.inner) * p.inner_stride + (i & ((1 << p.shift) - 1)) * 8;
    };
    uint4 v[kAhead];
    const int i0 = part * (kThreads * kAhead) + threadIdx.x;
    uint4* d[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kThreads;
        d[u] = nullptr;
        if (i >= p.vectors)
            continue;
        if constexpr (PACKED) {
            v[u] = reinterpret_cast<const uint4*>(p.kv.packed + from * page)[i];
            d[u] = reinterpret_cast<uint4*>(p.kv.packed + to * page) + i;
        } else {
            uint16_t* base = i < half ? p.kv.k : p.kv.v;
            const int64_t o = offset(i < half ? i : i - half);
            v[u] = *reinterpret_cast<const uint4*>(base + from * p.kv.page_stride + o);
            d[u] = reinterpret_cast<uint4*>(base + to * p.kv.page_stride + o);
        }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        if (d[u])
            *d[u] = v[u];
}

template <int DT>
cudaError_t launch_read(const ReadParams& p, cudaStream_t st)
{
    const dim3 grid((unsigned)((p.batch.tokens + kTokens - 1) / kTokens),
                    (unsigned)((2 * p.kv.heads * (p.kv.dim / 8) + kThreads - 1) / kThreads));
    return p.kv.packed ? launch_after(lbv_kv_read_kernel<DT, true>, grid, kThreads, 0, st, p)
                       : launch_after(lbv_kv_read_kernel<DT, false>, grid, kThreads, 0, st, p);
}

}  // namespace

cudaError_t launch_kv_read(const ReadParams& p, lbv_dtype dt, cudaStream_t st)
{
    return dt == LBV_F16 ? launch_read<LBV_F16>(p, st) : launch_read<LBV_BF16>(p, st);
}

cudaError_t launch_kv_keep(const lbv_batch& b, const KvView& kv, const uint64_t* kept, int32_t* left, cudaStream_t st)
{
    const dim3 grid((unsigned)b.requests, (unsigned)kv.heads);
    return kv.packed ? launch_after(lbv_kv_keep_kernel<true>, grid, kThreads, 0, st, b, kv, kept, left)
                     : launch_after(lbv_kv_keep_kernel<false>, grid, kThreads, 0, st, b, kv, kept, left);
}

cudaError_t launch_kv_copy_pages(const KvView& kv, const int32_t* src, const int32_t* dst, int count,
                                 cudaStream_t st)
{
    CopyParams p = {};
    p.kv = kv;
    p.src = src;
    p.dst = dst;
    const int64_t vectors = kv.packed ? kv4::page_bytes(kv) / 16 : (int64_t)2 * kv.heads * (kv.dim / 8) << kv.page_shift;
    p.vectors = (int)vectors;
    p.shift = kv.dim == 128 ? 4 : 3;
    const bool token_major = kv.head_stride <= kv.token_stride;
    p.inner = token_major ? kv.heads : 1 << kv.page_shift;
    p.inner_stride = token_major ? kv.head_stride : kv.token_stride;
    p.outer_stride = token_major ? kv.token_stride : kv.head_stride;
    p.parts = (int)((vectors + kThreads * kAhead - 1) / (kThreads * kAhead));
    const dim3 grid((unsigned)((int64_t)count * p.parts));
    return kv.packed ? launch_after(lbv_kv_copy_kernel<true>, grid, kThreads, 0, st, p)
                     : launch_after(lbv_kv_copy_kernel<false>, grid, kThreads, 0, st, p);
}

}  // namespace lbv

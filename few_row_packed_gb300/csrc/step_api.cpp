// step_api.cpp -- the C ABI of the operators around the verify matmul:
// argument checks, host handles and dispatch of the rotary append, the paged
// attention and the sampler.  Nothing here aborts or allocates device memory.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "attend_internal.h"
#include "step_internal.h"

namespace {

lbv_status fail(lbv_status st, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return lbv::set_error(st, buf);
}

lbv_status cuda_fail(cudaError_t e, const char* what)
{
    return fail(LBV_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t n)
{
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

bool is16(int dtype)
{
    return dtype == LBV_F16 || dtype == LBV_BF16;
}

size_t elem_size(int dtype)
{
    return dtype == LBV_F32 ? 4 : 2;
}

lbv_status check_batch(const char* fn, const lbv_batch* b)
{
    if (!b)
        return fail(LBV_ERR_INVALID_ARG, "%s: batch is NULL", fn);
    if (b->requests < 1 || b->requests > 4096 || b->tokens < 0)
        return fail(LBV_ERR_INVALID_ARG, "%s: requests=%d (1..4096) tokens=%d", fn, b->requests,
                    b->tokens);
    if (!b->q_start || !b->kv_len || !b->block_table || !aligned(b->q_start, 4) ||
        !aligned(b->kv_len, 4) || !aligned(b->block_table, 4))
        return fail(LBV_ERR_INVALID_ARG, "%s: null or misaligned batch array", fn);
    if (b->table_pages < 1 || b->table_stride < b->table_pages)
        return fail(LBV_ERR_INVALID_ARG, "%s: table_pages=%d table_stride=%d", fn, b->table_pages,
                    b->table_stride);
    return LBV_OK;
}

lbv_status check_rows(const char* fn, const char* what, const lbv_rows* r, int tokens)
{
    if (!r)
        return fail(LBV_ERR_INVALID_ARG, "%s: %s is NULL", fn, what);
    if (r->dtype != LBV_F16 && r->dtype != LBV_BF16 && r->dtype != LBV_F32)
        return fail(LBV_ERR_INVALID_ARG, "%s: %s has unknown dtype %d", fn, what, r->dtype);
    if (r->heads < 1 || r->heads > 65535)
        return fail(LBV_ERR_INVALID_ARG, "%s: %s has %d heads", fn, what, r->heads);
    if (tokens > 0 && (!r->data || !aligned(r->data, elem_size(r->dtype))))
        return fail(LBV_ERR_INVALID_ARG, "%s: %s is null or misaligned for its element type", fn,
                    what);
    return LBV_OK;
}

lbv_status check_cache(const char* fn, const lbv_kv_cache* c)
{
    if (!c)
        return fail(LBV_ERR_INVALID_ARG, "%s: cache is NULL", fn);
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != c->device)
        return fail(LBV_ERR_INVALID_ARG, "%s: current device %d is not the cache's %d", fn, dev,
                    c->device);
    return LBV_OK;
}

// The driver's tensor-map encoder, found once; NULL without a driver.
using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled()
{
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (EncodeTiled) nullptr;
        }
        return (EncodeTiled)p;
    }();
    return fn;
}

// Boxes of 64 elements of one head by min(page_size, 64) slots of one page, in
// 128-byte rows swizzled as ldmatrix and tcgen05 read them.
bool make_map(const lbv::KvView& v, lbv_dtype dtype, void* base, CUtensorMap* map)
{
    const EncodeTiled fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t page = (cuuint64_t)1 << v.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)v.dim, page, (cuuint64_t)v.heads, (cuuint64_t)v.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)v.token_stride * 2, (cuuint64_t)v.head_stride * 2,
                                   (cuuint64_t)v.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(page < 64 ? page : 64), 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(map, dtype == LBV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// ---------------------------------------------------------------------------
// The paged cache

lbv_status lbv_kv_cache_create(void* k, void* v, int pages, int page_size, int heads, int head_dim,
                               int64_t page_stride, int64_t token_stride, int64_t head_stride,
                               lbv_dtype dtype, lbv_kv_cache** out)
{
    const char* fn = "lbv_kv_cache_create";
    lbv::set_error(LBV_OK, "");
    if (!out)
        return fail(LBV_ERR_INVALID_ARG, "%s: out is NULL", fn);
    *out = nullptr;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16))
        return fail(LBV_ERR_INVALID_ARG, "%s: k or v is null or not 16-byte aligned", fn);
    if (!is16(dtype))
        return fail(LBV_ERR_INVALID_ARG, "%s: unknown cache dtype %d", fn, (int)dtype);
    if (pages < 1 || heads < 1 || heads > 65535)
        return fail(LBV_ERR_INVALID_ARG, "%s: pages=%d heads=%d", fn, pages, heads);
    if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
        return fail(LBV_ERR_UNSUPPORTED, "%s: page_size %d (a power of two, 8..1024)", fn,
                    page_size);
    if (head_dim != 64 && head_dim != 128)
        return fail(LBV_ERR_UNSUPPORTED, "%s: head_dim %d (64 or 128)", fn, head_dim);
    // the dimensions may come in any order but do not overlap: sorted by
    // stride, each holds the extent of the ones inside it
    int64_t st[3] = {page_stride, token_stride, head_stride};
    int64_t ext[3] = {pages, page_size, heads};
    for (int i = 0; i < 3; ++i) {
        if (st[i] < head_dim || st[i] % 8 != 0 || st[i] >= (int64_t)1 << 38)
            return fail(LBV_ERR_INVALID_ARG,
                        "%s: strides (%lld, %lld, %lld) are multiples of 8, at least head_dim", fn,
                        (long long)page_stride, (long long)token_stride, (long long)head_stride);
        for (int j = i; j > 0 && st[j] < st[j - 1]; --j) {
            const int64_t a = st[j], e = ext[j];
            st[j] = st[j - 1], ext[j] = ext[j - 1];
            st[j - 1] = a, ext[j - 1] = e;
        }
    }
    int64_t inner = head_dim;
    for (int i = 0; i < 3; ++i) {
        if (ext[i] > 1 && st[i] < inner)
            return fail(LBV_ERR_INVALID_ARG, "%s: strides (%lld, %lld, %lld) overlap", fn,
                        (long long)page_stride, (long long)token_stride, (long long)head_stride);
        // (an extent of 2^62 elements and more is no device's, and would pass 64 bits)
        if (ext[i] > 1 && st[i] > (((int64_t)1 << 62) - inner) / (ext[i] - 1))
            return fail(LBV_ERR_INVALID_ARG, "%s: strides (%lld, %lld, %lld) of %d pages, %d slots, %d heads", fn,
                        (long long)page_stride, (long long)token_stride, (long long)head_stride, pages,
                        page_size, heads);
        inner = st[i] * (ext[i] - 1) + inner;
    }
    lbv_kv_cache* c = new (std::nothrow) lbv_kv_cache();
    if (!c)
        return fail(LBV_ERR_INVALID_ARG, "%s: out of host memory", fn);
    int shift = 0;
    while ((1 << shift) < page_size)
        ++shift;
    c->view = {static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), page_stride, token_stride,
               head_stride, pages, shift, heads, head_dim};
    c->dtype = dtype;
    c->sms = 0;
    if (cudaGetDevice(&c->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&c->sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
        cudaGetLastError();
        c->device = -1;
    }
    c->maps = c->device >= 0 && make_map(c->view, dtype, k, &c->kmap) &&
              make_map(c->view, dtype, v, &c->vmap);
    if (c->device >= 0 && !c->maps) {
        delete c;
        return fail(LBV_ERR_CUDA, "%s: the driver has no tensor map for this layout", fn);
    }
    *out = c;
    return LBV_OK;
}

lbv_status lbv_kv_cache_destroy(lbv_kv_cache* cache)
{
    delete cache;
    return LBV_OK;
}

// ---------------------------------------------------------------------------
// Rotary positions

lbv_status lbv_rope_frequencies(int rot_dim, double base, lbv_rope_scaling scaling, double factor,
                                double trained, double low, double high, double* freqs)
{
    const char* fn = "lbv_rope_frequencies";
    lbv::set_error(LBV_OK, "");
    if (!freqs || rot_dim < 2 || rot_dim % 2 != 0 || !(base > 0) || !std::isfinite(base))
        return fail(LBV_ERR_INVALID_ARG, "%s: freqs NULL, rot_dim=%d or base=%g", fn, rot_dim,
                    base);
    if (scaling != LBV_ROPE_NONE && scaling != LBV_ROPE_LINEAR && scaling != LBV_ROPE_BY_PARTS)
        return fail(LBV_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, (int)scaling);
    if (scaling != LBV_ROPE_NONE && !(factor > 0 && std::isfinite(factor)))
        return fail(LBV_ERR_INVALID_ARG, "%s: factor=%g", fn, factor);
    if (scaling == LBV_ROPE_BY_PARTS && !(trained > 0 && low < high))
        return fail(LBV_ERR_INVALID_ARG, "%s: trained=%g low=%g high=%g", fn, trained, low, high);
    const double two_pi = 6.283185307179586476925;
    for (int j = 0; j < rot_dim / 2; ++j) {
        double f = std::pow(base, -2.0 * j / rot_dim);
        if (scaling == LBV_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == LBV_ROPE_BY_PARTS) {
            const double g = std::fmin(std::fmax((trained * f / two_pi - low) / (high - low), 0.0), 1.0);
            f *= (1.0 - g) / factor + g;
        }
        freqs[j] = f;
    }
    return LBV_OK;
}

lbv_status lbv_rope_create(const double* freqs, int rot_dim, lbv_rope_layout layout, float factor,
                           lbv_rope** out)
{
    const char* fn = "lbv_rope_create";
    lbv::set_error(LBV_OK, "");
    if (!out)
        return fail(LBV_ERR_INVALID_ARG, "%s: out is NULL", fn);
    *out = nullptr;
    if (!freqs || rot_dim < 8 || rot_dim > lbv::kMaxRot || rot_dim % 8 != 0)
        return fail(LBV_ERR_INVALID_ARG, "%s: freqs NULL or rot_dim=%d (a multiple of 8, 8..%d)",
                    fn, rot_dim, lbv::kMaxRot);
    if (layout != LBV_ROPE_HALF && layout != LBV_ROPE_INTERLEAVED)
        return fail(LBV_ERR_INVALID_ARG, "%s: unknown layout %d", fn, (int)layout);
    if (!std::isfinite(factor))
        return fail(LBV_ERR_INVALID_ARG, "%s: factor=%g", fn, (double)factor);
    for (int j = 0; j < rot_dim / 2; ++j)
        if (!std::isfinite(freqs[j]))
            return fail(LBV_ERR_INVALID_ARG, "%s: frequency %d is not finite", fn, j);
    lbv_rope* r = new (std::nothrow) lbv_rope();
    if (!r)
        return fail(LBV_ERR_INVALID_ARG, "%s: out of host memory", fn);
    const double two_pi = 6.283185307179586476925;
    for (int j = 0; j < rot_dim / 2; ++j) {
        // fraction of a turn per position in [0, 1), then in 2^-64 turns
        double t = freqs[j] / two_pi;
        t -= std::floor(t);
        const double s = std::ldexp(t, 64);
        r->turns[j] = s >= 18446744073709551616.0 ? 0 : (uint64_t)s;
    }
    r->rot = rot_dim;
    r->layout = layout;
    r->factor = factor;
    *out = r;
    return LBV_OK;
}

lbv_status lbv_rope_destroy(lbv_rope* rope)
{
    delete rope;
    return LBV_OK;
}

lbv_status lbv_rope_append(const lbv_rope* rope, const lbv_batch* batch, const lbv_kv_cache* cache,
                           const lbv_rows* q, const lbv_rows* k, const lbv_rows* v,
                           const lbv_rows* q_out, const int32_t* positions, lbv_stream stream)
{
    const char* fn = "lbv_rope_append";
    lbv::set_error(LBV_OK, "");
    if (!rope)
        return fail(LBV_ERR_INVALID_ARG, "%s: rope is NULL", fn);
    lbv_status st = check_batch(fn, batch);
    if (st == LBV_OK)
        st = check_rows(fn, "k", k, batch->tokens);
    if (st == LBV_OK)
        st = check_rows(fn, "v", v, batch->tokens);
    if (st == LBV_OK && (q || q_out)) {
        st = check_rows(fn, "q", q, batch->tokens);
        if (st == LBV_OK)
            st = check_rows(fn, "q_out", q_out, batch->tokens);
    }
    if (st == LBV_OK)
        st = check_cache(fn, cache);
    if (st != LBV_OK)
        return st;
    if (k->dtype != v->dtype || (q && q->dtype != k->dtype))
        return fail(LBV_ERR_INVALID_ARG, "%s: q, k and v have different dtypes", fn);
    if (q && (q_out->dtype != cache->dtype || q_out->heads != q->heads))
        return fail(LBV_ERR_INVALID_ARG, "%s: q_out is not of the cache's dtype with q's heads", fn);
    if (k->heads != cache->view.heads || v->heads != cache->view.heads)
        return fail(LBV_ERR_INVALID_ARG, "%s: k has %d and v %d heads, the cache %d", fn, k->heads,
                    v->heads, cache->view.heads);
    if (rope->rot > cache->view.dim)
        return fail(LBV_ERR_UNSUPPORTED, "%s: rot_dim %d exceeds head_dim %d", fn, rope->rot,
                    cache->view.dim);
    if (!aligned(positions, 4))
        return fail(LBV_ERR_INVALID_ARG, "%s: positions misaligned", fn);
    if (batch->tokens == 0)
        return LBV_OK;
    lbv::RopeParams p;
    const lbv_rows* rows[3] = {q, k, v};
    bool vec = true;        // 4-element loads of every row, 4-element stores of q_out
    for (int i = 0; i < 3; ++i) {
        const lbv_rows* r = rows[i];
        p.src[i] = r ? r->data : nullptr;
        p.src_token[i] = r ? r->token_stride : 0;
        p.src_head[i] = r ? r->head_stride : 0;
        vec = vec && (!r || (aligned(r->data, 4 * elem_size(r->dtype)) &&
                             r->token_stride % 4 == 0 && r->head_stride % 4 == 0));
    }
    p.q_out = q_out ? static_cast<uint16_t*>(q_out->data) : nullptr;
    p.out_token = q_out ? q_out->token_stride : 0;
    p.out_head = q_out ? q_out->head_stride : 0;
    vec = vec && (!q_out || (aligned(q_out->data, 8) && p.out_token % 4 == 0 && p.out_head % 4 == 0));
    for (int j = 0; j < rope->rot / 2; ++j)
        p.turns[j] = rope->turns[j];
    p.batch = *batch;
    p.kv = cache->view;
    p.positions = positions;
    p.q_heads = q ? q->heads : 0;
    p.rot = rope->rot;
    p.factor = rope->factor;
    const cudaError_t e = lbv::launch_rope_append(p, (lbv_dtype)k->dtype, cache->dtype,
                                                  rope->layout, vec, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return cuda_fail(e, "lbv_rope_append: launch");
    return LBV_OK;
}

// ---------------------------------------------------------------------------
// Attention over the paged cache

size_t lbv_attend_workspace_bytes(const lbv_kv_cache* cache, const lbv_batch* batch, int heads)
{
    if (!cache || !batch || heads < 1)
        return 0;
    const size_t rows = lbv::attend_rows_partial_floats(cache->view.dim, cache->sms);
    const size_t tiles = lbv::attend_tiles_partial_floats(cache->view.dim, cache->sms);
    return lbv::kAttendPartial + (rows > tiles ? rows : tiles) * sizeof(float);
}

// lbv_attend, by the name `fn`; copies >= 0: the test of the bounded waits.
static lbv_status attend(const char* fn, const lbv_kv_cache* cache, const lbv_batch* batch, const lbv_rows* q,
                         const lbv_rows* out, float scale, int window, const uint64_t* tree, float* lse,
                         void* workspace, size_t workspace_bytes, int copies, lbv_stream stream)
{
    lbv::set_error(LBV_OK, "");
    lbv_status st = check_batch(fn, batch);
    if (st == LBV_OK)
        st = check_rows(fn, "q", q, batch->tokens);
    if (st == LBV_OK)
        st = check_rows(fn, "out", out, batch->tokens);
    if (st == LBV_OK)
        st = check_cache(fn, cache);
    if (st != LBV_OK)
        return st;
    if (q->dtype != cache->dtype || out->dtype != cache->dtype)
        return fail(LBV_ERR_INVALID_ARG, "%s: q or out is not of the cache's dtype", fn);
    if (q->heads != out->heads || q->heads % cache->view.heads != 0)
        return fail(LBV_ERR_INVALID_ARG, "%s: %d query and %d output heads over %d cache heads", fn,
                    q->heads, out->heads, cache->view.heads);
    if (!std::isfinite(scale) || window < 0)
        return fail(LBV_ERR_INVALID_ARG, "%s: scale=%g window=%d", fn, (double)scale, window);
    if (!aligned(tree, 8) || !aligned(lse, 4))
        return fail(LBV_ERR_INVALID_ARG, "%s: tree or lse misaligned", fn);
    if (batch->tokens == 0)
        return LBV_OK;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < lbv_attend_workspace_bytes(cache, batch, q->heads))
        return fail(LBV_ERR_WORKSPACE, "%s: workspace NULL, not 256-byte aligned or %zu < %zu bytes",
                    fn, workspace_bytes, lbv_attend_workspace_bytes(cache, batch, q->heads));
    // the kernels count the costs of blocks of keys in 32 bits: an upper bound of theirs
    const double units = ((double)batch->tokens * q->heads / 16 + batch->requests * (double)cache->view.heads) *
                         ((double)batch->table_pages * (1 << cache->view.page_shift) / 32 + 32);
    if (units >= 4294967296.0)
        return fail(LBV_ERR_UNSUPPORTED, "%s: %d tokens over tables of %d pages are too many for one call",
                    fn, batch->tokens, batch->table_pages);
    lbv::AttendParams p;
    p.q = static_cast<const uint16_t*>(q->data);
    p.q_token = q->token_stride;
    p.q_head = q->head_stride;
    p.out = static_cast<uint16_t*>(out->data);
    p.out_token = out->token_stride;
    p.out_head = out->head_stride;
    p.lse = lse;
    p.tree = tree;
    p.scale_log2 = scale * 1.44269504088896341f;
    p.window = window < (1 << 30) ? window : 0;    // no context is that long
    p.heads = q->heads;
    p.group = q->heads / cache->view.heads;
    // the reciprocal rounded up at 31 + ceil(log2 group) bits divides all rows below 2^31
    for (p.group_shift = 0; (1ll << p.group_shift) < p.group; ++p.group_shift) {
    }
    p.group_mul = (uint32_t)(((1ull << (31 + p.group_shift)) + p.group - 1) / p.group);
    p.q_wide = aligned(q->data, 16) && q->token_stride % 8 == 0 && q->head_stride % 8 == 0;
    p.batch = *batch;
    p.kv = cache->view;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    p.status = reinterpret_cast<unsigned*>(ws);
    p.counters = reinterpret_cast<unsigned*>(ws + lbv::kAttendCounters);
    p.items = ws + lbv::kAttendItems;
    p.partial = reinterpret_cast<float*>(ws + lbv::kAttendPartial);
    p.wait_limit = copies < 0 ? lbv::kAttendWaitLimit : lbv::kAttendTestLimit;
    p.first_copies = copies < 0 ? ~0u : (unsigned)copies;
    // both kernels are right for every length
    const auto launch = lbv::attend_average_rows(p) <= 16 ? lbv::launch_attend_rows : lbv::launch_attend_tiles;
    const cudaError_t e = launch(p, cache->kmap, cache->vmap, cache->dtype, cache->sms,
                                 (cudaStream_t)stream);
    if (e != cudaSuccess)
        return cuda_fail(e, "lbv_attend: launch");
    return LBV_OK;
}

lbv_status lbv_attend(const lbv_kv_cache* cache, const lbv_batch* batch, const lbv_rows* q,
                      const lbv_rows* out, float scale, int window, const uint64_t* tree,
                      float* lse, void* workspace, size_t workspace_bytes, lbv_stream stream)
{
    return attend("lbv_attend", cache, batch, q, out, scale, window, tree, lse, workspace, workspace_bytes, -1,
                  stream);
}

lbv_status lbv_attend_test_wait(const lbv_kv_cache* cache, const lbv_batch* batch, const lbv_rows* q,
                                const lbv_rows* out, float scale, int window, const uint64_t* tree,
                                float* lse, void* workspace, size_t workspace_bytes, int copies,
                                lbv_stream stream)
{
    const char* fn = "lbv_attend_test_wait";
    if (copies < 0)
        return fail(LBV_ERR_INVALID_ARG, "%s: copies=%d", fn, copies);
    return attend(fn, cache, batch, q, out, scale, window, tree, lse, workspace, workspace_bytes, copies,
                  stream);
}

lbv_status lbv_attend_status(void* workspace)
{
    const char* fn = "lbv_attend_status";
    lbv::set_error(LBV_OK, "");
    if (!workspace)
        return fail(LBV_ERR_INVALID_ARG, "%s: workspace is NULL", fn);
    unsigned word = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess)
        e = cudaMemcpy(&word, workspace, sizeof word, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && word)
        e = cudaMemset(workspace, 0, lbv::kAttendItems);
    if (e != cudaSuccess)
        return cuda_fail(e, fn);
    if (word)
        return fail(LBV_ERR_TIMEOUT, "an attention kernel gave up waiting for its copies");
    return LBV_OK;
}

// ---------------------------------------------------------------------------
// Sampling

lbv_status lbv_sample(const void* logits, int M, int N, int64_t ld, lbv_dtype dtype,
                      const lbv_sample_rules* rules, const float* u, int32_t* token, float* prob,
                      lbv_stream stream)
{
    const char* fn = "lbv_sample";
    lbv::set_error(LBV_OK, "");
    if (dtype != LBV_F32 && dtype != LBV_F16 && dtype != LBV_BF16)
        return fail(LBV_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, (int)dtype);
    if (M < 0 || M > (1 << 24) || N < 1 || (M > 1 && ld < N))
        return fail(LBV_ERR_INVALID_ARG, "%s: M=%d N=%d ld=%lld", fn, M, N, (long long)ld);
    if (!rules)
        return fail(LBV_ERR_INVALID_ARG, "%s: rules is NULL", fn);
    if (rules->temperature_last != 0 && rules->temperature_last != 1)
        return fail(LBV_ERR_INVALID_ARG, "%s: temperature_last=%d", fn, rules->temperature_last);
    const void* words[] = {u, token, prob, rules->temperature, rules->top_k, rules->top_p,
                           rules->min_p, rules->mask};
    for (const void* w : words)
        if (!aligned(w, 4))
            return fail(LBV_ERR_INVALID_ARG, "%s: a per-row array is misaligned", fn);
    if (rules->mask && M > 1 && rules->mask_ld < (N + 31) / 32)
        return fail(LBV_ERR_INVALID_ARG, "%s: mask_ld=%lld < %d words", fn,
                    (long long)rules->mask_ld, (N + 31) / 32);
    if (N > 1 << 23)        // sums of weights up to 2^40 stay below 2^64
        return fail(LBV_ERR_UNSUPPORTED, "%s: N=%d exceeds %d logits a row", fn, N, 1 << 23);
    // Up to 8 rows take 16 CTAs each (one row of 151936, top-k and top-p: 14.0 us, 17.0
    // with 8; 8 rows, top-p and min-p: 32.4 and 35.5); of more,
    // 8 CTAs each keep four on every SM.  Short rows take fewer, so that a thread still
    // has a few logits.
    int ctas = M <= 8 ? 16 : 8;
    while (ctas > 1 && N <= ctas * 1024)
        ctas /= 2;
    if (M == 0)
        return LBV_OK;
    if (!logits || !aligned(logits, elem_size(dtype)) || !u || !token)
        return fail(LBV_ERR_INVALID_ARG, "%s: null or misaligned logits, u or token", fn);
    lbv::SampleParams p;
    p.logits = logits;
    p.mask = rules->mask;
    p.u = u;
    p.temperature = rules->temperature;
    p.top_k = rules->top_k;
    p.top_p = rules->top_p;
    p.min_p = rules->min_p;
    p.token = token;
    p.prob = prob;
    p.ld = ld;
    p.mask_ld = rules->mask_ld;
    p.N = N;
    p.ctas = ctas;
    p.slice = ((N + ctas - 1) / ctas + 31) / 32 * 32;
    p.temperature_last = rules->temperature_last;
    const cudaError_t e = lbv::launch_sample(p, M, dtype, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return cuda_fail(e, "lbv_sample: launch");
    return LBV_OK;
}

// step_internal.h -- the operators around the verify matmul (rotary append,
// paged attention, sampling): host objects, launch parameters and launchers
// shared by step_api.cpp and the kernels' files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/lbv.h"

namespace lbv {

// Records `message` ("" clears it) as the thread's last error; returns st.
lbv_status set_error(lbv_status st, const char* message);

// A paged cache as the kernels see it (strides in elements).
struct KvView {
    uint16_t* k;
    uint16_t* v;
    int64_t page_stride, token_stride, head_stride;
    int pages, page_shift, heads, dim;
    uint8_t* packed;                 // a cache of 4 bits (kv4.cuh), else NULL
};

// Frequencies of a rotation in 2^-64 turns per position.
constexpr int kMaxRot = 128;

struct RopeParams {
    uint64_t turns[kMaxRot / 2];
    const void* src[3];              // q, k, v rows
    int64_t src_token[3], src_head[3];
    uint16_t* q_out;                 // NULL: no queries
    int64_t out_token, out_head;
    lbv_batch batch;
    KvView kv;
    const int32_t* positions;        // NULL: cache positions
    int q_heads;                     // 0 without queries
    int rot;
    float factor;
};

cudaError_t launch_rope_append(const RopeParams& p, lbv_dtype src, lbv_dtype dst,
                               lbv_rope_layout layout, bool vec, cudaStream_t st);

// The append to a cache of 4 bits (append4.cu).
cudaError_t launch_rope_append4(const RopeParams& p, lbv_dtype src, lbv_dtype dst,
                                lbv_rope_layout layout, bool vec, cudaStream_t st);

struct ReadParams {
    lbv_batch batch;
    KvView kv;
    uint16_t* out[2];                // k, v rows; one may be NULL
    int64_t out_token[2], out_head[2];
    int wide;                        // rows are 16-byte aligned
};

cudaError_t launch_kv_read(const ReadParams& p, lbv_dtype dt, cudaStream_t st);
cudaError_t launch_kv_keep(const lbv_batch& b, const KvView& kv, const uint64_t* kept, int32_t* left,
                           cudaStream_t st);
cudaError_t launch_kv_copy_pages(const KvView& kv, const int32_t* src, const int32_t* dst, int count,
                                 cudaStream_t st);

struct SampleParams {
    const void* logits;              // [rows][ld]
    const uint32_t* mask;            // [rows][mask_ld] allowed-token bits, or NULL
    const float* u;                  // [rows]; the rest may be NULL
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;                  // [rows]
    float* prob;                     // [rows] or NULL
    int64_t ld, mask_ld;
    int N;
    int ctas, slice;                 // cluster size, logits per CTA (a multiple of 32)
    int temperature_last;
};

cudaError_t launch_sample(const SampleParams& p, int rows, lbv_dtype dt, cudaStream_t st);

#ifdef __CUDACC__
// These kernels launch while the one before them drains (launch_after); every thread
// waits for its end before it touches global memory.  (Against ordinary launches, us:
// the append for 64 requests 4.7 to 4.3, one token over 2,011 keys 12.3 to 11.4, a tree
// of 8 tokens 38.0 to 37.0.)
__device__ __forceinline__ void after_previous()
{
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

}  // namespace lbv

struct lbv_kv_cache {
    lbv::KvView view;
    lbv_dtype dtype;
    int device, sms;                 // -1: created without a device
    bool maps;                       // the tensor maps are there
    CUtensorMap kmap, vmap;          // boxes of 64 elements x the slots of a page in 64 keys
};

struct lbv_rope {
    uint64_t turns[lbv::kMaxRot / 2];
    int rot;
    lbv_rope_layout layout;
    float factor;
};

// attend_internal.h -- launch parameters of the attention kernels.
#pragma once

#include <cuda.h>

#include "step_internal.h"

namespace lbv {

struct AttendParams {
    const uint16_t* q;               // [tokens][heads][dim], strides in elements
    int64_t q_token, q_head;
    uint16_t* out;
    int64_t out_token, out_head;
    float* lse;                      // [tokens][heads], natural log, or NULL
    const uint64_t* tree;            // [tokens] or NULL
    float scale_log2;                // scale * log2(e)
    int window;                      // <= 0: none
    int heads, group;                // query heads, query heads per kv head
    uint32_t group_mul;              // row / group = (2 row * group_mul >> 32) >> group_shift
    int group_shift;
    int q_wide;                      // q rows are 16-byte aligned
    lbv_batch batch;
    KvView kv;
    // workspace
    unsigned* status;                // error bits
    unsigned* counters;              // one per CTA, zero between calls
    float* partial;                  // slots of partial results
    void* items;                     // one JoinItem per CTA where they are joined apart, else NULL
    unsigned wait_limit;             // clocks until a wait gives up
    unsigned first_copies;           // test only: copies that the first CTA makes (~0u: all)
};

constexpr unsigned kAttendWaitLimit = 1u << 31;  // about a second
constexpr unsigned kAttendTestLimit = 1u << 20;  // half a millisecond

constexpr int kAttendMaxCtas = 608;              // CTAs of a launch (152 SMs x 4), and counters
// Workspace: status word, counters, join items, partial results.
constexpr size_t kAttendCounters = 256;
constexpr size_t kAttendItems = kAttendCounters + kAttendMaxCtas * sizeof(unsigned);
constexpr size_t kAttendPartial = kAttendItems + kAttendMaxCtas * 32;

// Rows (new token times query head of a group) of an average request, whose
// lengths the host does not know.
inline int64_t attend_average_rows(const AttendParams& p)
{
    return ((int64_t)p.batch.tokens + p.batch.requests - 1) / p.batch.requests * p.group;
}

// p.items is where join items go if the launch joins apart.
cudaError_t launch_attend_rows(const AttendParams& p, const CUtensorMap& kmap,
                               const CUtensorMap& vmap, lbv_dtype dt, int sms, cudaStream_t st);
cudaError_t launch_attend_tiles(const AttendParams& p, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, lbv_dtype dt, int sms, cudaStream_t st);
// Joins apart (attend_join.cu): when, and the launch for slots of slot_rows rows.
bool attend_joins_apart(const AttendParams& p, int tile_rows, int ctas);
cudaError_t launch_attend_join(const AttendParams& p, lbv_dtype dt, int slot_rows, int ctas,
                               cudaStream_t st);
// Floats of workspace the launches need for partial results.
size_t attend_rows_partial_floats(int dim, int sms);
size_t attend_tiles_partial_floats(int dim, int sms);

}  // namespace lbv

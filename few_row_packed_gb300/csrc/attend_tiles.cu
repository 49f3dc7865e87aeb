// attend_tiles.cu -- the tensor-memory attention over a cache of 16 bits.
#include "attend_tiles.cuh"

namespace lbv {

cudaError_t launch_attend_tiles(const AttendParams& p, const CUtensorMap& kmap,
                                const CUtensorMap& vmap, lbv_dtype dt, int sms, cudaStream_t st)
{
    return launch_tiles<false>(p, kmap, vmap, dt, sms, st);
}

size_t attend_tiles_partial_floats(int dim, int sms)
{
    return (size_t)2 * (sms < kAttendMaxCtas ? sms : kAttendMaxCtas) * kRows * (dim + 3);
}

}  // namespace lbv

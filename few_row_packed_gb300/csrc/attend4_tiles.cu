// attend4_tiles.cu -- the tensor-memory attention over a cache of 4 bits.
#include "attend_tiles.cuh"

namespace lbv {

cudaError_t launch_attend4_tiles(const AttendParams& p, const CUtensorMap& kmap,
                                 const CUtensorMap& vmap, lbv_dtype dt, int sms, cudaStream_t st)
{
    return launch_tiles<true>(p, kmap, vmap, dt, sms, st);
}

}  // namespace lbv

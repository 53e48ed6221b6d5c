// Layer norm and RMS norm of fp32 rows, backward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_bwd_f32(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::bwd<float, float, true>(a, access, s, launches)
               : norm::bwd<float, float, false>(a, access, s, launches);
}

}  // namespace cce

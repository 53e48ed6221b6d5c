// Layer norm and RMS norm of fp32 rows, forward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_f32(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::fwd<float, float, true>(a, access, s, launches)
               : norm::fwd<float, float, false>(a, access, s, launches);
}

}  // namespace cce

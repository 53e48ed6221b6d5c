// Layer norm and RMS norm of fp32 rows with fp16 upstream gradients, backward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_bwd_f32_f16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::bwd<float, __half, true>(a, access, s, launches)
               : norm::bwd<float, __half, false>(a, access, s, launches);
}

}  // namespace cce

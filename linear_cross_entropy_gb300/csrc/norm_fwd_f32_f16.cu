// Layer norm and RMS norm of fp32 rows with fp16 results, forward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_f32_f16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::fwd<float, __half, true>(a, access, s, launches)
               : norm::fwd<float, __half, false>(a, access, s, launches);
}

}  // namespace cce

// Layer norm and RMS norm of fp32 rows with bf16 results, forward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_f32_bf16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::fwd<float, __nv_bfloat16, true>(a, access, s, launches)
               : norm::fwd<float, __nv_bfloat16, false>(a, access, s, launches);
}

}  // namespace cce

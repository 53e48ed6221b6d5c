// Layer norm and RMS norm of bf16 rows.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_bf16(const NormFwd& a, bool layer, bool wide, cudaStream_t s, int* launches) {
  return norm::fwd_any<__nv_bfloat16, __nv_bfloat16>(a, layer, wide, s, launches);
}

cudaError_t launch_norm_bwd_bf16(const NormBwd& a, bool layer, bool wide, cudaStream_t s, int* launches) {
  return norm::bwd_any<__nv_bfloat16, __nv_bfloat16>(a, layer, wide, s, launches);
}

}  // namespace cce

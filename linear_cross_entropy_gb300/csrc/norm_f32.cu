// Layer norm and RMS norm of fp32 rows, with fp32 or 16-bit results.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_f32(const NormFwd& a, int y_type, bool layer, bool wide, cudaStream_t s, int* launches) {
  if (y_type == CCE_BF16) return norm::fwd_any<float, __nv_bfloat16>(a, layer, wide, s, launches);
  if (y_type == CCE_F16) return norm::fwd_any<float, __half>(a, layer, wide, s, launches);
  return norm::fwd_any<float, float>(a, layer, wide, s, launches);
}

cudaError_t launch_norm_bwd_f32(const NormBwd& a, int y_type, bool layer, bool wide, cudaStream_t s, int* launches) {
  if (y_type == CCE_BF16) return norm::bwd_any<float, __nv_bfloat16>(a, layer, wide, s, launches);
  if (y_type == CCE_F16) return norm::bwd_any<float, __half>(a, layer, wide, s, launches);
  return norm::bwd_any<float, float>(a, layer, wide, s, launches);
}

}  // namespace cce

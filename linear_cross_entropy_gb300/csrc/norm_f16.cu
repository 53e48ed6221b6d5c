// Layer norm and RMS norm of fp16 rows.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_f16(const NormFwd& a, bool layer, bool wide, cudaStream_t s, int* launches) {
  return norm::fwd_any<__half, __half>(a, layer, wide, s, launches);
}

cudaError_t launch_norm_bwd_f16(const NormBwd& a, bool layer, bool wide, cudaStream_t s, int* launches) {
  return norm::bwd_any<__half, __half>(a, layer, wide, s, launches);
}

}  // namespace cce

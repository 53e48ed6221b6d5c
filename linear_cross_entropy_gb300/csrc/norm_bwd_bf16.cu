// Layer norm and RMS norm of bf16 rows, backward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_bwd_bf16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::bwd<__nv_bfloat16, __nv_bfloat16, true>(a, access, s, launches)
               : norm::bwd<__nv_bfloat16, __nv_bfloat16, false>(a, access, s, launches);
}

}  // namespace cce

// Layer norm and RMS norm of bf16 rows, forward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_bf16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::fwd<__nv_bfloat16, __nv_bfloat16, true>(a, access, s, launches)
               : norm::fwd<__nv_bfloat16, __nv_bfloat16, false>(a, access, s, launches);
}

}  // namespace cce

// Layer norm and RMS norm of fp16 rows, backward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_bwd_f16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::bwd<__half, __half, true>(a, access, s, launches)
               : norm::bwd<__half, __half, false>(a, access, s, launches);
}

}  // namespace cce

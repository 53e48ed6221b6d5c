// Layer norm and RMS norm of fp16 rows, forward.
#include "norm.cuh"

namespace cce {

cudaError_t launch_norm_fwd_f16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches) {
  return layer ? norm::fwd<__half, __half, true>(a, access, s, launches)
               : norm::fwd<__half, __half, false>(a, access, s, launches);
}

}  // namespace cce

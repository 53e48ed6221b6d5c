// The layers' GEMM with gelu in its epilogue.
#include "linear_gemm.cuh"

namespace cce {

cudaError_t prepare_linear_gemm_gelu() { return lin::prepare<CCE_ACT_GELU>(); }
cudaError_t launch_linear_gemm_gelu(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  return lin::launch<CCE_ACT_GELU>(a, pair, gated, units, s);
}

}  // namespace cce

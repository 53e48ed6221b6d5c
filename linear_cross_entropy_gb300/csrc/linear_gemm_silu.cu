// The layers' GEMM with silu in its epilogue.
#include "linear_gemm.cuh"

namespace cce {

cudaError_t prepare_linear_gemm_silu() { return lin::prepare<CCE_ACT_SILU>(); }
cudaError_t launch_linear_gemm_silu(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  return lin::launch<CCE_ACT_SILU>(a, pair, gated, units, s);
}

}  // namespace cce

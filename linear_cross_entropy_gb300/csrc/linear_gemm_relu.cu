// The layers' GEMM with relu in its epilogue.
#include "linear_gemm.cuh"

namespace cce {

cudaError_t prepare_linear_gemm_relu() { return lin::prepare<CCE_ACT_RELU>(); }
cudaError_t launch_linear_gemm_relu(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  return lin::launch<CCE_ACT_RELU>(a, pair, gated, units, s);
}

}  // namespace cce

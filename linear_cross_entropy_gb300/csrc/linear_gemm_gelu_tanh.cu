// The layers' GEMM with gelu_tanh in its epilogue.
#include "linear_gemm.cuh"

namespace cce {

cudaError_t prepare_linear_gemm_gelu_tanh() { return lin::prepare<CCE_ACT_GELU_TANH>(); }
cudaError_t launch_linear_gemm_gelu_tanh(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  return lin::launch<CCE_ACT_GELU_TANH>(a, pair, gated, units, s);
}

}  // namespace cce

// The layers' GEMM: the choice of its kernel by the activation, and the one without.
#include "linear_gemm.cuh"

namespace cce {

namespace {
__device__ int32_t linear_error;  // CCE_DEVERR_* of waits that ran out

// The wait of the GEMM's roles, on a barrier that nothing arrives on.
__global__ void wait_timeout_kernel(int32_t* error, uint64_t timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  mbar_init(&bar, 1);
  abort_flag = 0;
  fence_mbar_init();
  wait_bounded_long(&bar, 0, &abort_flag, error, timeout_ns);
}
}

cudaError_t launch_linear_wait_timeout(int32_t* error, uint64_t timeout_ns, cudaStream_t s) {
  wait_timeout_kernel<<<1, 1, 0, s>>>(error, timeout_ns);
  return cudaGetLastError();
}

cudaError_t prepare_linear_gemm(int32_t** error) {
  cudaError_t e = lin::prepare<CCE_ACT_NONE>();
  if (e == cudaSuccess) e = prepare_linear_gemm_relu();
  if (e == cudaSuccess) e = prepare_linear_gemm_gelu();
  if (e == cudaSuccess) e = prepare_linear_gemm_gelu_tanh();
  if (e == cudaSuccess) e = prepare_linear_gemm_silu();
  void* p = nullptr;
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&p, linear_error);
  *error = static_cast<int32_t*>(p);
  return e;
}

int linear_pair_units(int sms) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
  cfg.blockDim = dim3(lin::THREADS);
  cfg.dynamicSmemBytes = lin::SHARED;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, lin::linear_kernel<true, false, CCE_ACT_NONE, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_linear_gemm(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  // the activation is that of all products of a launch; behind partial sums it is for the joins
  switch (a.p[0].splits > 1 ? CCE_ACT_NONE : a.p[0].e.act) {
    case CCE_ACT_RELU: return launch_linear_gemm_relu(a, pair, gated, units, s);
    case CCE_ACT_GELU: return launch_linear_gemm_gelu(a, pair, gated, units, s);
    case CCE_ACT_GELU_TANH: return launch_linear_gemm_gelu_tanh(a, pair, gated, units, s);
    case CCE_ACT_SILU: return launch_linear_gemm_silu(a, pair, gated, units, s);
    default: return lin::launch<CCE_ACT_NONE>(a, pair, gated, units, s);
  }
}

cudaError_t take_linear_error(int32_t* word, cudaStream_t s) {
  const int32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, linear_error, sizeof zero, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *word != 0) {
    e = cudaMemcpyToSymbolAsync(linear_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace cce

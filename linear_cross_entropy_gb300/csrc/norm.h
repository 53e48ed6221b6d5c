// Layer norm and RMS norm: arguments of the kernels and their launchers, shared
// by the entry points (norm_api.cu) and the per-type translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace cce {

// Start of row n in elements: rows in runs of `inner` at row_stride, the runs
// at outer_stride.
struct RowMap {
  int64_t row_stride, outer_stride;
  int inner;

  __device__ __forceinline__ int64_t at(int64_t n) const {
    if (n < inner) return n * row_stride;
    const int o = static_cast<int>(n) / inner;
    return o * outer_stride + (n - static_cast<int64_t>(o) * inner) * row_stride;
  }
};

struct NormFwd {
  const void* x;
  RowMap xm;
  const void* w;  // may be null
  const void* b;  // may be null
  void* y;
  float* mean;  // may be null
  float* rstd;  // may be null
  int p_type, N, D;
  float eps, offset;
  int sms;  // of the device
  // With Access::REALIGNED:
  int shift;      // elements by which y starts behind a vector's start
  int64_t x_end;  // elements from x to the end of its last row
};

struct NormBwd {
  const void* dy;
  RowMap gm;
  const void* x;
  RowMap xm;
  const void* w;  // may be null
  const float* mean;
  const float* rstd;
  void* dx;       // may be null
  void* dw;       // may be null
  void* db;       // may be null
  float* part_w;  // [parts][D]
  float* part_b;  // [parts][D]
  int p_type, N, D;
  float offset;
  int sms;  // of the device
  // With Access::REALIGNED:
  int shift;              // elements by which dx starts behind a vector's start
  int64_t x_end, dy_end;  // elements from x and dy to the end of their last rows
  bool cluster = false;  // the launcher's: the grid is one cluster that writes dw and db
};

// Blocks whose partial parameter gradients are added at the end, at most.
constexpr int NORM_MAX_PARTS = 304;

// How rows are read and written: in aligned vectors of 16 bytes of x, which rows
// consist of; in such vectors, whose elements a row's start shifts, alike in every
// matrix; the same, shifted otherwise in some; by elements.
enum class Access { WIDE, SHIFTED, REALIGNED, SINGLE };

// The pair of types is one the entry points allow; `layer` picks layer norm or RMS norm.
cudaError_t launch_norm_fwd_bf16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_fwd_f16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_fwd_f32(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_fwd_f32_bf16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_fwd_f32_f16(const NormFwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_bwd_bf16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_bwd_f16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_bwd_f32(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_bwd_f32_bf16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches);
cudaError_t launch_norm_bwd_f32_f16(const NormBwd& a, bool layer, Access access, cudaStream_t s, int* launches);

}  // namespace cce

// Entry points of layer norm and RMS norm (include/cce_ops.h): argument checks,
// workspace layout, choice of the access width, launches.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/cce_ops.h"
#include "internal.h"
#include "norm.h"

namespace cce {
namespace {

// Columns from which rows are taken in vectors wherever they start: a row's two partial vectors are then the lesser
// part.  With rows shifted otherwise in one matrix than in another, fp16, 16 x 1,023 x 2,049 without every last token:
// forward and backward of a layer norm 58 and 111 us, by elements 80 and 235; 1,029 x 1,001 7.2 and 10.7, by elements
// 5.9 and 14.1.
constexpr int64_t SHIFTED_MIN = 64;
constexpr int64_t LIMIT = int64_t(1) << 31;

struct Rows {
  int64_t inner, row_stride, outer_stride;
};

int type_bytes(int t) { return t == CCE_F32 ? 4 : 2; }
bool type_ok(int t) { return t == CCE_F32 || t == CCE_F16 || t == CCE_BF16; }
bool pair_ok(int x, int y) { return type_ok(x) && type_ok(y) && (x == y || x == CCE_F32); }
bool multiple(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }
bool sizes_ok(int64_t N, int64_t D) { return N >= 0 && N < LIMIT && D >= 1 && D < LIMIT; }
bool rows_ok(const Rows& r) { return r.inner >= 1 && r.row_stride >= 0 && r.outer_stride >= 0; }

RowMap row_map(const Rows& r) {
  return RowMap{r.row_stride, r.outer_stride, static_cast<int>(std::min(r.inner, LIMIT - 1))};
}

// Whether rows at p can be read and written `vec` elements at a time.
bool rows_wide(const void* p, const Rows& r, int type, int vec) {
  return multiple(p, std::min(16, vec * type_bytes(type))) && r.row_stride % vec == 0 && r.outer_stride % vec == 0;
}
// Elements by which p lies behind a vector's start.
int shift_of(const void* p, int type, int vec) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) / static_cast<uintptr_t>(type_bytes(type))) & (vec - 1);
}
// Whether every row of a matrix starts at its index times D, modulo vec, from an
// aligned base, and the last one lies behind all others.
bool rows_shifted(const void* p, const Rows& r, int type, int vec, int64_t N, int64_t D) {
  return shift_of(p, type, vec) == 0 && r.inner >= N &&
         (N <= 1 || (r.row_stride >= D && (r.row_stride - D) % vec == 0));
}
// Elements to the end of the last row in memory.
int64_t rows_end(const Rows& r, int64_t N, int64_t D) {
  if (N == 0) return 0;
  const int64_t inner = std::min(r.inner, N), runs = N / inner, rest = N % inner;
  const int64_t whole = (runs - 1) * r.outer_stride + (inner - 1) * r.row_stride;
  return D + (rest > 0 ? std::max(whole, runs * r.outer_stride + (rest - 1) * r.row_stride) : whole);
}
bool param_wide(const void* p, int type, int vec) { return multiple(p, std::min(16, vec * type_bytes(type))); }

size_t part_bytes(int64_t N, int64_t D) {
  const size_t parts = static_cast<size_t>(std::max<int64_t>(1, std::min<int64_t>(NORM_MAX_PARTS, N)));
  return (parts * static_cast<size_t>(D) * sizeof(float) + 255) / 256 * 256;
}

cce_status status_of(cudaError_t e) { return e == cudaSuccess ? CCE_OK : CCE_ERR_CUDA; }

cce_status forward(const void* x, const Rows& xr, int x_type, const void* w, const void* b, int p_type, float offset,
                   int64_t N, int64_t D, float eps, void* y, int y_type, float* mean, float* rstd, bool layer,
                   void* stream) {
  if (!pair_ok(x_type, y_type) || !type_ok(p_type)) return CCE_ERR_ARG;
  if (!std::isfinite(eps) || eps < 0.0f || !std::isfinite(offset)) return CCE_ERR_ARG;
  if (!sizes_ok(N, D) || !rows_ok(xr)) return CCE_ERR_SHAPE;
  if (N > 0 && (!x || !y)) return CCE_ERR_NULL;
  if (!multiple(x, type_bytes(x_type)) || !multiple(y, type_bytes(y_type)) || !multiple(w, type_bytes(p_type)) ||
      !multiple(b, type_bytes(p_type)) || !multiple(mean, 4) || !multiple(rstd, 4))
    return CCE_ERR_ALIGN;
  int sms = 0;
  const cce_status st = static_cast<cce_status>(device_ready(&sms));
  if (st != CCE_OK) return st;
  const int vec = 16 / type_bytes(x_type);
  const Rows dense{N, D, 0};
  const Access access = D % vec == 0 && rows_wide(x, xr, x_type, vec) && rows_wide(y, dense, y_type, vec) &&
                                param_wide(w, p_type, vec) && param_wide(b, p_type, vec)
                            ? Access::WIDE
                        : D < SHIFTED_MIN ? Access::SINGLE
                        : rows_shifted(x, xr, x_type, vec, N, D) && rows_shifted(y, dense, y_type, vec, N, D)
                            ? Access::SHIFTED
                            : Access::REALIGNED;
  const NormFwd a{x,
                  row_map(xr),
                  w,
                  b,
                  y,
                  mean,
                  rstd,
                  p_type,
                  static_cast<int>(N),
                  static_cast<int>(D),
                  eps,
                  offset,
                  sms,
                  shift_of(y, y_type, vec),
                  rows_end(xr, N, D)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  const auto launch = x_type == CCE_BF16  ? launch_norm_fwd_bf16
                      : x_type == CCE_F16   ? launch_norm_fwd_f16
                      : y_type == CCE_F32   ? launch_norm_fwd_f32
                      : y_type == CCE_BF16  ? launch_norm_fwd_f32_bf16
                                            : launch_norm_fwd_f32_f16;
  const cudaError_t e = launch(a, layer, access, s, &launches);
  count_launches(launches);
  return status_of(e);
}

cce_status backward(const void* dy, const Rows& gr, int y_type, const void* x, const Rows& xr, int x_type,
                    const void* w, int p_type, float offset, const float* mean, const float* rstd, int64_t N,
                    int64_t D, void* dx, void* dw, void* db, void* workspace, size_t ws_bytes, bool layer,
                    void* stream) {
  if (!pair_ok(x_type, y_type) || !type_ok(p_type) || !std::isfinite(offset)) return CCE_ERR_ARG;
  if (!sizes_ok(N, D) || !rows_ok(gr) || !rows_ok(xr)) return CCE_ERR_SHAPE;
  const bool params = dw || db;
  if (N > 0 && (!dy || !x || !rstd || (layer && !mean))) return CCE_ERR_NULL;
  if (N > 0 && params && !workspace) return CCE_ERR_NULL;
  if (!multiple(dy, type_bytes(y_type)) || !multiple(x, type_bytes(x_type)) || !multiple(dx, type_bytes(x_type)) ||
      !multiple(w, type_bytes(p_type)) || !multiple(dw, type_bytes(p_type)) || !multiple(db, type_bytes(p_type)) ||
      !multiple(mean, 4) || !multiple(rstd, 4) || !multiple(workspace, 16))
    return CCE_ERR_ALIGN;
  if (N > 0 && params && ws_bytes < 2 * part_bytes(N, D)) return CCE_ERR_WORKSPACE;
  int sms = 0;
  const cce_status st = static_cast<cce_status>(device_ready(&sms));
  if (st != CCE_OK) return st;
  const int vec = 16 / type_bytes(x_type);
  const Rows dense{N, D, 0};
  const Access access = D % vec == 0 && rows_wide(x, xr, x_type, vec) && rows_wide(dy, gr, y_type, vec) &&
                                rows_wide(dx, dense, x_type, vec) && param_wide(w, p_type, vec)
                            ? Access::WIDE
                        : D < SHIFTED_MIN ? Access::SINGLE
                        : rows_shifted(x, xr, x_type, vec, N, D) && rows_shifted(dy, gr, y_type, vec, N, D) &&
                                rows_shifted(dx, dense, x_type, vec, N, D)
                            ? Access::SHIFTED
                            : Access::REALIGNED;
  char* ws = static_cast<char*>(workspace);
  const NormBwd a{dy,
                  row_map(gr),
                  x,
                  row_map(xr),
                  w,
                  mean,
                  rstd,
                  dx,
                  dw,
                  db,
                  reinterpret_cast<float*>(ws),
                  reinterpret_cast<float*>(ws ? ws + part_bytes(N, D) : nullptr),
                  p_type,
                  static_cast<int>(N),
                  static_cast<int>(D),
                  offset,
                  sms,
                  shift_of(dx ? dx : x, x_type, vec),
                  rows_end(xr, N, D),
                  rows_end(gr, N, D)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  const auto launch = x_type == CCE_BF16  ? launch_norm_bwd_bf16
                      : x_type == CCE_F16   ? launch_norm_bwd_f16
                      : y_type == CCE_F32   ? launch_norm_bwd_f32
                      : y_type == CCE_BF16  ? launch_norm_bwd_f32_bf16
                                            : launch_norm_bwd_f32_f16;
  const cudaError_t e = launch(a, layer, access, s, &launches);
  count_launches(launches);
  return status_of(e);
}

}  // namespace
}  // namespace cce

using namespace cce;

extern "C" {

int cce_ops_abi_version(void) { return 100; }

cce_status cce_layer_norm_forward(const void* x, int64_t x_inner, int64_t x_row_stride, int64_t x_outer_stride,
                                  int x_type, const void* weight, const void* bias, int p_type, int64_t N, int64_t D,
                                  float eps, void* y, int y_type, float* mean, float* rstd, void* stream) {
  return forward(x, Rows{x_inner, x_row_stride, x_outer_stride}, x_type, weight, bias, p_type, 0.0f, N, D, eps, y,
                 y_type, mean, rstd, true, stream);
}

cce_status cce_rms_norm_forward(const void* x, int64_t x_inner, int64_t x_row_stride, int64_t x_outer_stride,
                                int x_type, const void* weight, int p_type, float weight_offset, int64_t N, int64_t D,
                                float eps, void* y, int y_type, float* rstd, void* stream) {
  return forward(x, Rows{x_inner, x_row_stride, x_outer_stride}, x_type, weight, nullptr, p_type, weight_offset, N,
                 D, eps, y, y_type, nullptr, rstd, false, stream);
}

cce_status cce_layer_norm_backward(const void* grad_y, int64_t g_inner, int64_t g_row_stride, int64_t g_outer_stride,
                                   int y_type, const void* x, int64_t x_inner, int64_t x_row_stride,
                                   int64_t x_outer_stride, int x_type, const void* weight, int p_type,
                                   const float* mean, const float* rstd, int64_t N, int64_t D, void* grad_x,
                                   void* grad_weight, void* grad_bias, void* workspace, size_t ws_bytes,
                                   void* stream) {
  return backward(grad_y, Rows{g_inner, g_row_stride, g_outer_stride}, y_type, x,
                  Rows{x_inner, x_row_stride, x_outer_stride}, x_type, weight, p_type, 0.0f, mean, rstd, N, D, grad_x,
                  grad_weight, grad_bias, workspace, ws_bytes, true, stream);
}

cce_status cce_rms_norm_backward(const void* grad_y, int64_t g_inner, int64_t g_row_stride, int64_t g_outer_stride,
                                 int y_type, const void* x, int64_t x_inner, int64_t x_row_stride,
                                 int64_t x_outer_stride, int x_type, const void* weight, int p_type,
                                 float weight_offset, const float* rstd, int64_t N, int64_t D, void* grad_x,
                                 void* grad_weight, void* workspace, size_t ws_bytes, void* stream) {
  return backward(grad_y, Rows{g_inner, g_row_stride, g_outer_stride}, y_type, x,
                  Rows{x_inner, x_row_stride, x_outer_stride}, x_type, weight, p_type, weight_offset, nullptr, rstd,
                  N, D, grad_x, grad_weight, nullptr, workspace, ws_bytes, false, stream);
}

size_t cce_norm_backward_workspace_bytes(int64_t N, int64_t D) {
  return sizes_ok(N, D) ? 2 * part_bytes(N, D) : 0;
}

}  // extern "C"

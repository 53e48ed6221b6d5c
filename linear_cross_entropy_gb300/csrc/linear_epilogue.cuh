// What happens to an accumulator of a layer on its way out (LinEpilogue), for a
// thread that holds consecutive rows j of one output column i.
#pragma once

#include "activation.cuh"
#include "elements.cuh"
#include "linear.h"

namespace cce {

template <int ACT, int M>
__device__ __forceinline__ void activate_as(float (&z)[M]) {
#pragma unroll
  for (int u = 0; u < M; ++u) z[u] = activate<ACT>(z[u]);
}

// The activation is uniform over a launch: one branch for M values.
template <int M>
__device__ __forceinline__ void activate_all(int act, float (&z)[M]) {
  switch (act) {
    case CCE_ACT_RELU: activate_as<CCE_ACT_RELU>(z); break;
    case CCE_ACT_GELU: activate_as<CCE_ACT_GELU>(z); break;
    case CCE_ACT_GELU_TANH: activate_as<CCE_ACT_GELU_TANH>(z); break;
    case CCE_ACT_SILU: activate_as<CCE_ACT_SILU>(z); break;
    default: break;
  }
}

__device__ __forceinline__ float load_scalar(const void* p, int type, int64_t i) {
  float f[1];
  load_param<1>(p, type, i, f);
  return f[0];
}

// Rows j0 .. j0 + n - 1 (n <= M) of column i, all inside of the matrices.  z0:
// the product with x (gated: the gate's), z1: gated: the up projection's.
template <bool BF16, bool Y32, bool GATED, int M>
__device__ __forceinline__ void finish_column_as(const LinEpilogue& e, float bias, int i, int j0, int n,
                                                 float (&z0)[M], float (&z1)[M]) {
  float res[M];
  if (!GATED && e.res) {  // all loads in flight at once
#pragma unroll
    for (int u = 0; u < M; ++u) {
      if (u < n) {
        const int64_t at = static_cast<int64_t>(j0 + u) * e.res_pitch + i;
        res[u] = Y32 ? static_cast<const float*>(e.res)[at]
                     : from_bits16<BF16>(static_cast<const uint16_t*>(e.res)[at]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < M; ++u) z0[u] += bias;
  if (e.z[0]) {
#pragma unroll
    for (int u = 0; u < M; ++u) {
      if (u < n) {
        const int64_t at = static_cast<int64_t>(j0 + u) * e.z_pitch + i;
        static_cast<uint16_t*>(e.z[0])[at] = to_bits16<BF16>(z0[u]);
        if (GATED) static_cast<uint16_t*>(e.z[1])[at] = to_bits16<BF16>(z1[u]);
      }
    }
  }
  activate_all(e.act, z0);
#pragma unroll
  for (int u = 0; u < M; ++u) {
    if (u < n) {
      float y = z0[u];
      if (GATED) y *= z1[u];
      if (!GATED && e.res) y += res[u];
      const int64_t at = static_cast<int64_t>(j0 + u) * e.y_pitch + i;
      if (Y32) {
        static_cast<float*>(e.y)[at] = y;
      } else {
        static_cast<uint16_t*>(e.y)[at] = to_bits16<BF16>(y);
      }
    }
  }
}

template <bool GATED, int M>
__device__ __forceinline__ void finish_column(const LinEpilogue& e, bool bf16, float bias, int i, int j0, int n,
                                              float (&z0)[M], float (&z1)[M]) {
  if (e.y_type == CCE_F32) {
    if (bf16) {
      finish_column_as<true, true, GATED>(e, bias, i, j0, n, z0, z1);
    } else {
      finish_column_as<false, true, GATED>(e, bias, i, j0, n, z0, z1);
    }
  } else if (bf16) {
    finish_column_as<true, false, GATED>(e, bias, i, j0, n, z0, z1);
  } else {
    finish_column_as<false, false, GATED>(e, bias, i, j0, n, z0, z1);
  }
}

}  // namespace cce

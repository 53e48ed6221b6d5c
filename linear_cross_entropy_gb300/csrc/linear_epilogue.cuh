// What happens to an accumulator of a layer on its way out (LinEpilogue), for a
// thread that holds consecutive rows j of one output column i.
#pragma once

#include "activation.cuh"
#include "elements.cuh"
#include "linear.h"

#include <type_traits>

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

// Rows j0 .. j0 + n - 1 of column i, all inside of the matrices; n = M with FULL.
// z0: the product with x (gated: the gate's), z1: gated: the up projection's.
template <bool BF16, bool Y32, bool GATED, bool FULL, int M>
__device__ __forceinline__ void finish_column_as(const LinEpilogue& e, float bias, int i, int j0, int n,
                                                 float (&z0)[M], float (&z1)[M]) {
  using Y = typename std::conditional<Y32, float, uint16_t>::type;
  float res[M];
  if (!GATED && e.res) {  // all loads in flight at once
    const Y* p = static_cast<const Y*>(e.res) + static_cast<int64_t>(j0) * e.res_pitch + i;
#pragma unroll
    for (int u = 0; u < M; ++u, p += e.res_pitch) {
      if (FULL || u < n) {
        if constexpr (Y32) {
          res[u] = *p;
        } else {
          res[u] = from_bits16<BF16>(*p);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < M; ++u) z0[u] += bias;
  if (e.z[0]) {
    uint16_t* p = static_cast<uint16_t*>(e.z[0]) + static_cast<int64_t>(j0) * e.z_pitch + i;
    uint16_t* q = static_cast<uint16_t*>(e.z[1]) + static_cast<int64_t>(j0) * e.z_pitch + i;
#pragma unroll
    for (int u = 0; u < M; ++u, p += e.z_pitch, q += e.z_pitch) {
      if (FULL || u < n) {
        *p = to_bits16<BF16>(z0[u]);
        if (GATED) *q = to_bits16<BF16>(z1[u]);
      }
    }
  }
  activate_all(e.act, z0);
  Y* p = static_cast<Y*>(e.y) + static_cast<int64_t>(j0) * e.y_pitch + i;
#pragma unroll
  for (int u = 0; u < M; ++u, p += e.y_pitch) {
    if (FULL || u < n) {
      float y = z0[u];
      if (GATED) y *= z1[u];
      if (!GATED && e.res) y += res[u];
      if constexpr (Y32) {
        *p = y;
      } else {
        *p = to_bits16<BF16>(y);
      }
    }
  }
}

template <bool BF16, bool Y32, bool GATED, int M>
__device__ __forceinline__ void finish_column_of(const LinEpilogue& e, float bias, int i, int j0, int n, float (&z0)[M],
                                                 float (&z1)[M]) {
  if (M == 1 || n >= M) {
    finish_column_as<BF16, Y32, GATED, true>(e, bias, i, j0, n, z0, z1);
  } else {
    finish_column_as<BF16, Y32, GATED, false>(e, bias, i, j0, n, z0, z1);
  }
}

template <bool GATED, int M>
__device__ __forceinline__ void finish_column(const LinEpilogue& e, bool bf16, float bias, int i, int j0, int n,
                                              float (&z0)[M], float (&z1)[M]) {
  if (!GATED && e.y_type == CCE_F32) {
    if (bf16) {
      finish_column_of<true, true, GATED>(e, bias, i, j0, n, z0, z1);
    } else {
      finish_column_of<false, true, GATED>(e, bias, i, j0, n, z0, z1);
    }
  } else if (bf16) {
    finish_column_of<true, false, GATED>(e, bias, i, j0, n, z0, z1);
  } else {
    finish_column_of<false, false, GATED>(e, bias, i, j0, n, z0, z1);
  }
}

}  // namespace cce

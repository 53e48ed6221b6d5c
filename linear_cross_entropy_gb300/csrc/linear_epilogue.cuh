// What happens to a sum of products of a layer on its way out (LinEpilogue).
#pragma once

#include "activation.cuh"
#include "elements.cuh"
#include "linear.h"

namespace cce {

template <int ACT, int M>
__device__ __forceinline__ void activate_as(float (&z)[M]) {
#pragma unroll
  for (int u = 0; u + 1 < M; u += 2) activate_pair<ACT>(z[u], z[u + 1]);
  if constexpr (M % 2 != 0) {
    float none = 0.0f;
    activate_pair<ACT>(z[M - 1], none);
  }
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

// Column c of the sums of a gradient's parts: eight running sums of every eighth part, then those in order.
__device__ __forceinline__ void sum_columns(const LinSum& a, int c) {
  if (c >= a.N) return;
  float t[8] = {};
  const float* p = a.part + c;
  const int64_t n = a.N;
  int at = 0;
#pragma unroll 4
  for (; at + 8 <= a.parts; at += 8) {
#pragma unroll
    for (int v = 0; v < 8; ++v) t[v] += p[(at + v) * n];
  }
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    if (at + v < a.parts) t[v] += p[(at + v) * n];
  }
#pragma unroll
  for (int v = 1; v < 8; ++v) t[0] += t[v];
  store_param(a.db, a.type, c, t[0]);
}

template <typename T, int VEC>
__device__ __forceinline__ void put(void* base, int64_t at, const float (&f)[VEC]) {
  Vec<T, VEC> v;
  v.set(f);
  v.store(static_cast<T*>(base) + at);
}

template <int VEC>
__device__ __forceinline__ void put_kept(void* base, int64_t at, const float (&f)[VEC]) {
  Vec<__nv_bfloat16, VEC> v;
  v.zero();
#pragma unroll
  for (int u = 0; u < VEC; ++u) v.w[u / 2] |= to_kept16(f[u]) << (16 * (u & 1));
  v.store(static_cast<__nv_bfloat16*>(base) + at);
}

// Where row j of the residual starts.
__device__ __forceinline__ int64_t res_row(const LinEpilogue& e, int64_t j) {
  if (e.res_inner == 0) return j * e.res_pitch;
  const uint32_t n = static_cast<uint32_t>(j), run = n / static_cast<uint32_t>(e.res_inner);
  return run * e.res_outer + (n - run * static_cast<uint32_t>(e.res_inner)) * e.res_pitch;
}

// VEC neighbouring values i, ... of row j, all inside of the matrices, which VEC values of each start on their size.  z0:
// the product with x (gated: the gate's), z1: gated: the up projection's.  T: the operands' type.
template <typename T, bool GATED, int VEC>
__device__ __forceinline__ void finish_row(const LinEpilogue& e, int64_t j, int64_t i, float (&z0)[VEC],
                                           const float (&z1)[VEC]) {
  const bool y32 = !GATED && e.y_type == CCE_F32;
  if (!GATED && e.bias) {
    float b[VEC];
    load_param<VEC>(e.bias, e.bias_type, i, b);
#pragma unroll
    for (int u = 0; u < VEC; ++u) z0[u] += b[u];
  }
  if (e.z[0]) {
    const int64_t at = j * e.z_pitch + i;
    if (e.z_type == CCE_KEPT16) {
      put_kept(e.z[0], at, z0);
      if (GATED) put_kept(e.z[1], at, z1);
    } else {
      put<T>(e.z[0], at, z0);
      if (GATED) put<T>(e.z[1], at, z1);
    }
  }
  activate_all(e.act, z0);
  if (GATED) {
#pragma unroll
    for (int u = 0; u < VEC; ++u) z0[u] *= z1[u];
  } else if (e.res) {
    float r[VEC];
    load_param<VEC>(e.res, y32 ? CCE_F32 : ElemType<T>::id, res_row(e, j) + i, r);
#pragma unroll
    for (int u = 0; u < VEC; ++u) z0[u] += r[u];
  }
  if (y32) {
    put<float>(e.y, j * e.y_pitch + i, z0);
  } else {
    put<T>(e.y, j * e.y_pitch + i, z0);
  }
}

}  // namespace cce

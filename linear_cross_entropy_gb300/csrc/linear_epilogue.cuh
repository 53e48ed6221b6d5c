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

// Loads and stores of a column's rows, `pitch` bytes apart.  They are volatile so that
// they stay in order and each address is the last one and a pitch: with all addresses in
// registers at once the epilogue spilled.
__device__ __forceinline__ void store16(char* p, uint32_t v) {
  asm volatile("{\n\t.reg .b16 h, g;\n\tmov.b32 {h, g}, %1;\n\tst.global.b16 [%0], h;\n\t}" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void store16_high(char* p, uint32_t v) {
  asm volatile("{\n\t.reg .b16 h, g;\n\tmov.b32 {h, g}, %1;\n\tst.global.b16 [%0], g;\n\t}" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void store32(char* p, float v) {
  asm volatile("st.global.f32 [%0], %1;" ::"l"(p), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t load16(const char* p) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load32(const char* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// M values to rows of a 16-bit matrix, rounded to nearest even; the first n of them.
template <bool FULL, int M>
__device__ __forceinline__ void store_rows16(char* p, int64_t pitch, const uint32_t (&two)[(M + 1) / 2], int n) {
#pragma unroll
  for (int u = 0; u < M; ++u, p += pitch) {
    if (!FULL && u >= n) continue;
    if (u & 1) {
      store16_high(p, two[u / 2]);
    } else {
      store16(p, two[u / 2]);
    }
  }
}

template <int M>
__device__ __forceinline__ void put_rows16(void* base, int64_t pitch, int64_t at, bool bf16, const float (&f)[M], int n) {
  uint32_t two[(M + 1) / 2];
  if (bf16) {
#pragma unroll
    for (int u = 0; u < M; u += 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[u], u + 1 < M ? f[u + 1 < M ? u + 1 : u] : 0.0f);
      two[u / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int u = 0; u < M; u += 2) {
      const __half2 h = __floats2half2_rn(f[u], u + 1 < M ? f[u + 1 < M ? u + 1 : u] : 0.0f);
      two[u / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  char* p = static_cast<char*>(base) + at * 2;
  if (n >= M) {
    store_rows16<true, M>(p, pitch * 2, two, n);
  } else {
    store_rows16<false, M>(p, pitch * 2, two, n);
  }
}

template <int M>
__device__ __forceinline__ void put_rows32(void* base, int64_t pitch, int64_t at, const float (&f)[M], int n) {
  char* p = static_cast<char*>(base) + at * 4;
#pragma unroll
  for (int u = 0; u < M; ++u, p += pitch * 4) {
    if (u < n) store32(p, f[u]);
  }
}

// The residual's rows as they are in memory: loaded ahead of what they are added to.
template <int M>
struct Residual {
  uint32_t raw[M];

  __device__ __forceinline__ void load(const LinEpilogue& e, int i, int j0, int n) {
    const int64_t at = static_cast<int64_t>(j0) * e.res_pitch + i;
    if (e.y_type == CCE_F32) {
      const char* p = static_cast<const char*>(e.res) + at * 4;
#pragma unroll
      for (int u = 0; u < M; ++u, p += e.res_pitch * 4) raw[u] = u < n ? load32(p) : 0u;
    } else {
      const char* p = static_cast<const char*>(e.res) + at * 2;
#pragma unroll
      for (int u = 0; u < M; ++u, p += e.res_pitch * 2) raw[u] = u < n ? load16(p) : 0u;
    }
  }
  __device__ __forceinline__ void add_to(const LinEpilogue& e, bool bf16, float (&f)[M]) const {
    if (e.y_type == CCE_F32) {
#pragma unroll
      for (int u = 0; u < M; ++u) f[u] += __uint_as_float(raw[u]);
    } else if (bf16) {
#pragma unroll
      for (int u = 0; u < M; ++u) f[u] += __uint_as_float(raw[u] << 16);
    } else {
#pragma unroll
      for (int u = 0; u < M; ++u) f[u] += __half2float(__ushort_as_half(static_cast<uint16_t>(raw[u])));
    }
  }
};

// Rows j0 .. j0 + min(n, M) - 1 of column i, all inside of the matrices.  z0: the
// product with x (gated: the gate's), z1: gated: the up projection's; res: loaded if
// there is a residual.
template <bool GATED, int M>
__device__ __forceinline__ void finish_column(const LinEpilogue& e, bool bf16, float bias, int i, int j0, int n,
                                              float (&z0)[M], const float (&z1)[M], const Residual<M>& res) {
  if (!GATED && e.bias) {
#pragma unroll
    for (int u = 0; u < M; ++u) z0[u] += bias;
  }
  if (e.z[0]) {
    const int64_t at = static_cast<int64_t>(j0) * e.z_pitch + i;
    put_rows16(e.z[0], e.z_pitch, at, bf16, z0, n);
    if (GATED) put_rows16(e.z[1], e.z_pitch, at, bf16, z1, n);
  }
  activate_all(e.act, z0);
  if (GATED) {
#pragma unroll
    for (int u = 0; u < M; ++u) z0[u] *= z1[u];
  } else if (e.res) {
    res.add_to(e, bf16, z0);
  }
  const int64_t at = static_cast<int64_t>(j0) * e.y_pitch + i;
  if (!GATED && e.y_type == CCE_F32) {
    put_rows32(e.y, e.y_pitch, at, z0, n);
  } else {
    put_rows16(e.y, e.y_pitch, at, bf16, z0, n);
  }
}

}  // namespace cce

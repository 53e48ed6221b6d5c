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

// Loads and stores of a column's rows, a pitch apart.  They are volatile so that they
// stay in order and each address is the last one and a pitch: with all addresses in
// registers at once the epilogue spilled.
__device__ __forceinline__ void store16(char* p, uint32_t v) {
  asm volatile("{\n\t.reg .b16 h, g;\n\tmov.b32 {h, g}, %1;\n\tst.global.b16 [%0], h;\n\t}" ::"l"(p), "r"(v));
}
__device__ __forceinline__ void store16_high(char* p, uint32_t v) {
  asm volatile("{\n\t.reg .b16 h, g;\n\tmov.b32 {h, g}, %1;\n\tst.global.b16 [%0], g;\n\t}" ::"l"(p), "r"(v));
}
__device__ __forceinline__ void store32(char* p, float v) {
  asm volatile("st.global.f32 [%0], %1;" ::"l"(p), "f"(v));
}
__device__ __forceinline__ uint32_t load16(const char* p) {
  uint16_t v;
  asm volatile("ld.global.b16 %0, [%1];" : "=h"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load32(const char* p) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// A thread's place in the matrices of an epilogue, in registers: kernel parameters
// behind a run-time index cost a load for each use.
struct Column {
  char *y = nullptr, *z = nullptr;
  const char* res = nullptr;
  uint32_t y_step = 0, z_step = 0, res_step = 0;  // bytes from row to row
  float bias = 0.0f;
  int act = 0;
  bool bf16 = false, y32 = false, has_bias = false;

  template <bool GATED>
  __device__ __forceinline__ void start(const LinEpilogue& e, bool operands_bf16, int i, int j) {
    bf16 = operands_bf16;
    y32 = !GATED && e.y_type == CCE_F32;
    act = e.act;
    const uint32_t bytes = y32 ? 4 : 2;
    y_step = static_cast<uint32_t>(e.y_pitch) * bytes;
    y = static_cast<char*>(e.y) + static_cast<int64_t>(j) * y_step + static_cast<int64_t>(i) * bytes;
    if (e.z[0]) {
      z_step = static_cast<uint32_t>(e.z_pitch) * 2;
      z = static_cast<char*>(e.z[0]) + static_cast<int64_t>(j) * z_step + static_cast<int64_t>(i) * 2;
    }
    if (!GATED && e.res) {
      res_step = static_cast<uint32_t>(e.res_pitch) * bytes;
      res = static_cast<const char*>(e.res) + static_cast<int64_t>(j) * res_step + static_cast<int64_t>(i) * bytes;
    }
    has_bias = !GATED && e.bias;
    if (has_bias) bias = load_scalar(e.bias, e.bias_type, i);
  }
  __device__ __forceinline__ void skip(uint32_t rows) {
    y += static_cast<uint64_t>(rows) * y_step;
    if (z) z += static_cast<uint64_t>(rows) * z_step;
    if (res) res += static_cast<uint64_t>(rows) * res_step;
  }
};

// M values to rows of a 16-bit matrix, rounded to nearest even; the first n of them.
template <bool FULL, int M>
__device__ __forceinline__ void store_rows16(char* p, uint32_t step, const uint32_t (&two)[(M + 1) / 2], int n) {
#pragma unroll
  for (int u = 0; u < M; ++u, p += step) {
    if (!FULL && u >= n) continue;
    if (u & 1) {
      store16_high(p, two[u / 2]);
    } else {
      store16(p, two[u / 2]);
    }
  }
}

template <int M>
__device__ __forceinline__ void put_rows16(char* p, uint32_t step, bool bf16, const float (&f)[M], int n) {
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
  if (n >= M) {
    store_rows16<true, M>(p, step, two, n);
  } else {
    store_rows16<false, M>(p, step, two, n);
  }
}

template <int M>
__device__ __forceinline__ void put_rows32(char* p, uint32_t step, const float (&f)[M], int n) {
#pragma unroll
  for (int u = 0; u < M; ++u, p += step) {
    if (u < n) store32(p, f[u]);
  }
}

// The residual's rows as they are in memory: loaded ahead of what they are added to.
template <int M>
struct Residual {
  uint32_t raw[M];

  __device__ __forceinline__ void load(const Column& c, int n) {
    const char* p = c.res;
    if (c.y32) {
#pragma unroll
      for (int u = 0; u < M; ++u, p += c.res_step) raw[u] = u < n ? load32(p) : 0u;
    } else {
#pragma unroll
      for (int u = 0; u < M; ++u, p += c.res_step) raw[u] = u < n ? load16(p) : 0u;
    }
  }
  __device__ __forceinline__ void add_to(const Column& c, float (&f)[M]) const {
    if (c.y32) {
#pragma unroll
      for (int u = 0; u < M; ++u) f[u] += __uint_as_float(raw[u]);
    } else if (c.bf16) {
#pragma unroll
      for (int u = 0; u < M; ++u) f[u] += __uint_as_float(raw[u] << 16);
    } else {
#pragma unroll
      for (int u = 0; u < M; ++u) f[u] += __half2float(__ushort_as_half(static_cast<uint16_t>(raw[u])));
    }
  }
};

// min(n, M) rows from the column's place on.  z0: the product with x (gated: the
// gate's), z1: gated: the up projection's; res: loaded if there is a residual.
template <bool GATED, int M>
__device__ __forceinline__ void finish_column(const LinEpilogue& e, const Column& c, int n, float (&z0)[M], const float (&z1)[M],
                                              const Residual<M>& res) {
  if (!GATED && c.has_bias) {
#pragma unroll
    for (int u = 0; u < M; ++u) z0[u] += c.bias;
  }
  if (c.z) {
    put_rows16(c.z, c.z_step, c.bf16, z0, n);
    if (GATED) put_rows16(c.z + (static_cast<char*>(e.z[1]) - static_cast<char*>(e.z[0])), c.z_step, c.bf16, z1, n);
  }
  activate_all(c.act, z0);
  if (GATED) {
#pragma unroll
    for (int u = 0; u < M; ++u) z0[u] *= z1[u];
  } else if (c.res) {
    res.add_to(c, z0);
  }
  if (!GATED && c.y32) {
    put_rows32(c.y, c.y_step, z0, n);
  } else {
    put_rows16(c.y, c.y_step, c.bf16, z0, n);
  }
}

}  // namespace cce

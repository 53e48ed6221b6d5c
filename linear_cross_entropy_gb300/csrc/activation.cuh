// Activations of the layers in front of the head, and storing their results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/cce_layers.h"

namespace cce {

// Logistic function; exact at both ends: e^-z is infinite or 0 there.
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float GELU_C = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float GELU_C3 = 0.035677408136300125f;  // 0.044715 sqrt(2 / pi)
constexpr float SQRT_HALF = 0.7071067811865476f;
constexpr float INV_SQRT_2PI = 0.3989422804014327f;

// z / (1 + e^-z), -0 at minus infinity as the limit is.
__device__ __forceinline__ float silu(float z) { return z == -INFINITY ? -0.0f : z * logistic(z); }

// 0.5 (1 + tanh u) = logistic(2 u), u = c (z + 0.044715 z^3).  u overflows to an infinity of z's sign at most.
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  const float u = z * fmaf(GELU_C3 * z, z, GELU_C);
  return logistic(2.0f * u);
}
__device__ __forceinline__ float gelu_gate(float z) { return 0.5f * erfcf(-SQRT_HALF * z); }

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == CCE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if constexpr (ACT == CCE_ACT_GELU) return z == -INFINITY ? -0.0f : z * gelu_gate(z);
  if constexpr (ACT == CCE_ACT_GELU_TANH) return z == -INFINITY ? -0.0f : z * gelu_tanh_gate(z);
  if constexpr (ACT == CCE_ACT_SILU) return silu(z);
  return z;
}

// f(z) and f'(z).  The terms z f'' of infinite z vanish: z is held within +-200, where every gate is 0 or 1 to the last bit.
template <int ACT>
__device__ __forceinline__ float2 activate_both(float z) {
  if constexpr (ACT == CCE_ACT_RELU) return make_float2(z < 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : z != z ? z : 0.0f);
  if constexpr (ACT == CCE_ACT_GELU) {
    const float c = z > 200.0f ? 200.0f : z < -200.0f ? -200.0f : z;
    const float g = gelu_gate(c);
    return make_float2(activate<ACT>(z), fmaf(c * INV_SQRT_2PI, __expf(-0.5f * c * c), g));
  }
  if constexpr (ACT == CCE_ACT_GELU_TANH) {
    const float c = z > 200.0f ? 200.0f : z < -200.0f ? -200.0f : z;
    const float s = gelu_tanh_gate(c);
    // d logistic(2 u) = 2 s (1 - s) du
    const float du = fmaf(3.0f * GELU_C3 * c, c, GELU_C);
    return make_float2(activate<ACT>(z), fmaf(2.0f * c * s * (1.0f - s), du, s));
  }
  if constexpr (ACT == CCE_ACT_SILU) {
    const float c = z > 200.0f ? 200.0f : z < -200.0f ? -200.0f : z;
    const float s = logistic(c);
    return make_float2(silu(z), s * fmaf(c, 1.0f - s, 1.0f));
  }
  return make_float2(z, 1.0f);
}

// One of the 16-bit operand types from fp32, to nearest even.
template <bool BF16>
__device__ __forceinline__ uint16_t to_bits16(float f) {
  if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  return __half_as_ushort(__float2half_rn(f));
}
template <bool BF16>
__device__ __forceinline__ float from_bits16(uint16_t b) {
  if constexpr (BF16) return __uint_as_float(static_cast<uint32_t>(b) << 16);
  return __half2float(__ushort_as_half(b));
}

}  // namespace cce

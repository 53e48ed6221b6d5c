// Activations of the layers in front of the head, and storing their results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/cce_layers.h"

namespace cce {

constexpr float GELU_C = 0.7978845608028654f;     // sqrt(2 / pi)
constexpr float GELU_C3 = 0.035677408136300125f;  // 0.044715 sqrt(2 / pi)
constexpr float INV_SQRT_2PI = 0.3989422804014327f;
constexpr float LOG2_E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Logistic function; exact at both ends: e^-z is infinite or 0 there.
__device__ __forceinline__ float logistic(float z) { return reciprocal_fast(1.0f + exp2_fast(-LOG2_E * z)); }

// 0.5 (1 + tanh u) = logistic(2 u), u = c (z + 0.044715 z^3).  u overflows to an infinity of z's sign at most.
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  const float u = z * fmaf(GELU_C3 * z, z, GELU_C);
  return logistic(2.0f * u);
}

// The normal distribution function by the rational approximation 7.1.26 of Abramowitz and Stegun's Handbook of
// Mathematical Functions: erfc(x) = t (a1 + t (a2 + ...)) e^(-x^2), t = 1 / (1 + p x), x >= 0, within 1.5e-7; here
// x = |z| / sqrt(2), and Phi(z) is half of it below 0 and one less that above.  CUDA's erfcf takes twice the
// instructions: with it 65,536 x 2,048 x 8,192 took 2,171 us and not 1,374.
__device__ __forceinline__ float gelu_gate(float z) {
  const float m = fabsf(z);
  const float t = reciprocal_fast(fmaf(0.3275911f * 0.70710678f, m, 1.0f));
  float s = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  s = fmaf(s, t, 0.5f * 1.421413741f);
  s = fmaf(s, t, 0.5f * -0.284496736f);
  s = fmaf(s, t, 0.5f * 0.254829592f);
  s = s * t * exp2_fast(-0.5f * LOG2_E * m * m);
  return z < 0.0f ? s : 1.0f - s;
}

// -0 at minus infinity, as the limit is.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == CCE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if constexpr (ACT == CCE_ACT_GELU) return z == -INFINITY ? -0.0f : z * gelu_gate(z);
  if constexpr (ACT == CCE_ACT_GELU_TANH) return z == -INFINITY ? -0.0f : z * gelu_tanh_gate(z);
  if constexpr (ACT == CCE_ACT_SILU) return z == -INFINITY ? -0.0f : z * logistic(z);
  return z;
}

// f(z) and f'(z).  The terms z f'' of infinite z vanish: z is held within +-200, where every gate is 0 or 1 to the last bit.
template <int ACT>
__device__ __forceinline__ float2 activate_both(float z) {
  if constexpr (ACT == CCE_ACT_RELU) return make_float2(z < 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : z != z ? z : 0.0f);
  if constexpr (ACT == CCE_ACT_GELU) {
    const float c = z > 200.0f ? 200.0f : z < -200.0f ? -200.0f : z;
    const float g = gelu_gate(c);
    return make_float2(activate<ACT>(z), fmaf(c * INV_SQRT_2PI, exp2_fast(-0.5f * LOG2_E * c * c), g));
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
    return make_float2(activate<ACT>(z), s * fmaf(c, 1.0f - s, 1.0f));
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

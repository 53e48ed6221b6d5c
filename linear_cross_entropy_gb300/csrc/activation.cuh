// Activations of the layers in front of the head, and storing their results.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/cce_layers.h"
#include "elements.cuh"

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
// instructions.
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

// Every activation but relu vanishes towards minus infinity: from -1e30 on, where its gate is 0, z counts as that, or it
// would be infinity times 0.  (As a choice between results the compiler makes a branch of it, and 16 activations
// of a thread run one after another: gelu took 1,600 cycles and not some 300.)  A NaN stays one.
__device__ __forceinline__ float from_below(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(-1e30f));
  return r;
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == CCE_ACT_RELU) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if constexpr (ACT == CCE_ACT_NONE) return z;
  z = from_below(z);
  if constexpr (ACT == CCE_ACT_GELU) return z * gelu_gate(z);
  if constexpr (ACT == CCE_ACT_GELU_TANH) return z * gelu_tanh_gate(z);
  return z * logistic(z);
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

// ------------------------------------------------------------- in pairs
// The forward's activations, two at a time in packed fp32: reciprocals and powers of two share one slow unit of an SM,
// so that only one of them is taken there.

// 1 / (1 + 2^x).  2^x is the Taylor polynomial of degree 6 of 2^f, |f| <= 1/2 (within 1.2e-7), times 2^n; at x = 128
// and above it is infinite and the result 0.
__device__ __forceinline__ Pair logistic_of_power(Pair x) {
  constexpr float ROUND = 12582912.0f;  // 1.5 2^23: adding it leaves the nearest integer in the low bits
  const float2 v = x.get();
  const Pair c = Pair::of(fminf(fmaxf(v.x, -126.0f), 128.0f), fminf(fmaxf(v.y, -126.0f), 128.0f));
  const Pair t = add(c, Pair::both(ROUND));
  const Pair f = add(c, mul(add(t, Pair::both(-ROUND)), Pair::both(-1.0f)));
  Pair s = fma(Pair::both(1.5403530e-4f), f, Pair::both(1.3333558e-3f));
  s = fma(s, f, Pair::both(9.6181291e-3f));
  s = fma(s, f, Pair::both(5.5504109e-2f));
  s = fma(s, f, Pair::both(2.4022651e-1f));
  s = fma(s, f, Pair::both(6.9314718e-1f));
  const float2 p = fma(s, f, Pair::both(1.0f)).get(), n = t.get();
  const auto scaled = [](float m, float e) { return __uint_as_float(__float_as_uint(e) * (1u << 23) + __float_as_uint(m)); };
  const float2 d = add(Pair::of(scaled(p.x, n.x), scaled(p.y, n.y)), Pair::both(1.0f)).get();
  return Pair::of(reciprocal_fast(d.x), reciprocal_fast(d.y));
}

// The normal distribution function by formula 7.1.28 of the Handbook: erfc(x) = (1 + a1 x + ... + a6 x^6)^-16, x >= 0,
// within 3e-7.
__device__ __forceinline__ Pair normal_pair(Pair z) {
  constexpr float R = 0.70710678f;  // x = R |z|, and the powers of R go into the coefficients
  const float2 v = z.get();
  const Pair m = Pair::of(fabsf(v.x), fabsf(v.y));
  Pair s = fma(Pair::both(0.0000430638f * R * R * R * R * R * R), m, Pair::both(0.0002765672f * R * R * R * R * R));
  s = fma(s, m, Pair::both(0.0001520143f * R * R * R * R));
  s = fma(s, m, Pair::both(0.0092705272f * R * R * R));
  s = fma(s, m, Pair::both(0.0422820123f * R * R));
  s = fma(s, m, Pair::both(0.0705230784f * R));
  s = fma(s, m, Pair::both(1.0f));
  s = mul(s, s);
  s = mul(s, s);
  s = mul(s, s);
  const float2 d = mul(s, s).get();
  const float lo = 0.5f * reciprocal_fast(d.x), hi = 0.5f * reciprocal_fast(d.y);
  return Pair::of(v.x < 0.0f ? lo : 1.0f - lo, v.y < 0.0f ? hi : 1.0f - hi);
}

template <int ACT>
__device__ __forceinline__ void activate_pair(float& lo, float& hi) {
  if constexpr (ACT == CCE_ACT_NONE || ACT == CCE_ACT_RELU) {
    lo = activate<ACT>(lo);
    hi = activate<ACT>(hi);
  } else {
    const Pair z = Pair::of(from_below(lo), from_below(hi));
    Pair gate;
    if constexpr (ACT == CCE_ACT_GELU) gate = normal_pair(z);
    if constexpr (ACT == CCE_ACT_SILU) gate = logistic_of_power(mul(z, Pair::both(-LOG2_E)));
    if constexpr (ACT == CCE_ACT_GELU_TANH)
      gate = logistic_of_power(
          mul(z, fma(mul(z, z), Pair::both(-2.0f * LOG2_E * GELU_C3), Pair::both(-2.0f * LOG2_E * GELU_C))));
    const float2 y = mul(z, gate).get();
    lo = y.x;
    hi = y.y;
  }
}

// ---------------------------------------------------------------- 16 bits
// CCE_KEPT16 (include/cce_layers.h): times 2^-96 an fp32 value's exponent is that of the format, whose subnormals are
// then fp32's; what remains is to round off 14 bits.
__device__ __forceinline__ uint32_t to_kept16(float f) {
  const uint32_t b = __float_as_uint(f * 0x1p-96f), m = b & 0x7fffffffu;
  const uint32_t r = min((m + 0x2000u) >> 14, 0x7e00u);
  return (f == f ? r : 0x7fffu) | (b >> 16 & 0x8000u);
}
__device__ __forceinline__ float from_kept16(uint32_t h) {
  const uint32_t m = h & 0x7fffu;
  const float f = __uint_as_float(m << 14) * 0x1p96f;
  return copysignf(m < 0x7e00u ? f : m == 0x7e00u ? INFINITY : NAN, __uint_as_float(h << 16));
}

// The largest magnitude, or NaN if there is one.
template <int N>
__device__ __forceinline__ float largest(const float (&f)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int x = 0; x + 1 < N; x += 2)
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(f[x]), "f"(f[x + 1]));
  if (N % 2) asm("max.NaN.abs.f32 %0, %1, %2, %2;" : "=f"(m) : "f"(m), "f"(f[N - 1]));
  return m;
}

// Pairs of values, the first in the low half.  Where none comes near the format's largest, two bits of exponent are 0
// and what lies below them moves up: 3 instructions a value and not 10.
template <int M>
__device__ __forceinline__ void to_kept16(const float (&f)[2 * M], uint32_t (&two)[M]) {
  if (largest(f) < 0x1p31f) {
#pragma unroll
    for (int x = 0; x < M; ++x) {
      const float2 scaled = mul(Pair::of(f[2 * x], f[2 * x + 1]), Pair::both(0x1p-96f)).get();
      const uint32_t lo = __float_as_uint(scaled.x), hi = __float_as_uint(scaled.y);
      two[x] = __byte_perm(((lo * 4u + 0x8000u) & 0x7fffffffu) | (lo & 0x80000000u),
                           ((hi * 4u + 0x8000u) & 0x7fffffffu) | (hi & 0x80000000u), 0x7632);
    }
  } else {
#pragma unroll
    for (int x = 0; x < M; ++x) two[x] = to_kept16(f[2 * x]) | to_kept16(f[2 * x + 1]) << 16;
  }
}
template <int VEC>
__device__ __forceinline__ void from_kept16(const uint32_t* two, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = from_kept16(two[0]);
  } else {
#pragma unroll
    for (int x = 0; x < VEC; ++x) {
      const int32_t up = static_cast<int32_t>(x & 1 ? two[x / 2] : two[x / 2] << 16);
      f[x] = __uint_as_float(static_cast<uint32_t>(up >> 2) & 0x9fffc000u) * 0x1p96f;
    }
    if (!(largest(f) < 0x1p32f)) {
#pragma unroll
      for (int x = 0; x < VEC; ++x) f[x] = from_kept16(two[x / 2] >> (16 * (x & 1)));
    }
  }
}

// 16-bit types that the layers write.
enum Bits16 { BITS_F16 = CCE_F16, BITS_BF16 = CCE_BF16, BITS_KEPT = CCE_KEPT16 };

// Pairs of values, the first in the low half; one branch for all of them.
template <int M>
__device__ __forceinline__ void to_bits16(int type, const float (&f)[2 * M], uint32_t (&two)[M]) {
  if (type == BITS_BF16) {
#pragma unroll
    for (int x = 0; x < M; ++x) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * x], f[2 * x + 1]);
      two[x] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else if (type == BITS_F16) {
#pragma unroll
    for (int x = 0; x < M; ++x) {
      const __half2 h = __floats2half2_rn(f[2 * x], f[2 * x + 1]);
      two[x] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
    to_kept16<M>(f, two);
  }
}

}  // namespace cce

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

// gelu from the normal distribution function Phi(-m) = e^(-m^2 / 2) P(m) / Q(m), m = |z|, which keeps its relative accuracy
// as it vanishes: P / Q is a rational fit to e^(m^2 / 2) Phi(-m) for 0 <= m <= 16, within 4.9e-7 of its value (least squares
// with weights moved to the largest errors; P(0) = 1/2), and m^2 / 2 is rounded, so that Phi is within (z^2 + 16) 2^-23 of
// itself.  (Forms of the Handbook of Mathematical Functions, 7.1.26 and 7.1.28, have an absolute bound: at z = -4 the shorter
// was off by 0.4% and at -6 by a quarter.)  Then z Phi(z) = max(z, 0) - m Phi(-m); from m = 16 on, where Phi(-m) is 0 in
// fp32, m counts as that.  Both passes take the same steps.  8,192 x 896 x 4,864 takes 50 us as it did by 7.1.28, and 77 for
// 75 where z is kept.
constexpr float GATE_P1 = 0.364253402f, GATE_P2 = 0.120802656f, GATE_P3 = 0.0173314139f;
constexpr float GATE_Q1 = 1.52637613f, GATE_Q2 = 0.959620535f, GATE_Q3 = 0.302628309f, GATE_Q4 = 0.0434475578f;
constexpr float GATE_END = 16.0f;

struct GeluTail {
  float m, power, phi;  // min(|z|, 16), e^(-m^2 / 2), Phi(-m)
};

__device__ __forceinline__ GeluTail gelu_tail(float z) {
  const float m = fminf(fabsf(z), GATE_END);
  const float p = fmaf(fmaf(fmaf(GATE_P3, m, GATE_P2), m, GATE_P1), m, 0.5f);
  const float q = fmaf(fmaf(fmaf(fmaf(GATE_Q4, m, GATE_Q3), m, GATE_Q2), m, GATE_Q1), m, 1.0f);
  const float e = exp2_fast(__fmul_rn(__fmul_rn(m, m), -0.5f * LOG2_E));
  return {m, e, __fmul_rn(__fmul_rn(p, e), reciprocal_fast(q))};
}

// max(z, 0); a NaN stays one.
__device__ __forceinline__ float positive_part(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(z), "f"(0.0f));
  return r;
}

// silu and tanh-gelu vanish towards minus infinity: from -1e30 on, where their gate is 0, z counts as that, or they
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
  if constexpr (ACT == CCE_ACT_GELU) {
    const GeluTail t = gelu_tail(z);
    return fmaf(-t.m, t.phi, positive_part(z));
  }
  z = from_below(z);
  if constexpr (ACT == CCE_ACT_GELU_TANH) return z * gelu_tanh_gate(z);
  return z * logistic(z);
}

// f(z) and f'(z).  The terms z f'' of infinite z vanish: z is held within +-200, where every gate is 0 or 1 to the last bit.
template <int ACT>
__device__ __forceinline__ float2 activate_both(float z) {
  if constexpr (ACT == CCE_ACT_RELU) return make_float2(z < 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : z != z ? z : 0.0f);
  if constexpr (ACT == CCE_ACT_GELU) {
    const float c = z > 200.0f ? 200.0f : z < -200.0f ? -200.0f : z;
    const GeluTail t = gelu_tail(z);
    return make_float2(fmaf(-t.m, t.phi, positive_part(z)),
                       fmaf(c * INV_SQRT_2PI, t.power, z < 0.0f ? t.phi : 1.0f - t.phi));
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
// The forward's activations, two at a time in packed fp32.  Reciprocals and powers of two share one slow unit of an SM:
// silu's and tanh-gelu's powers of two are not taken there.

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

// (P with its sign turned, so that the last step needs no negation.)
__device__ __forceinline__ Pair gelu_pair(float lo, float hi) {
  const Pair m = Pair::of(fminf(fabsf(lo), GATE_END), fminf(fabsf(hi), GATE_END));
  Pair p = fma(Pair::both(-GATE_P3), m, Pair::both(-GATE_P2));
  p = fma(p, m, Pair::both(-GATE_P1));
  p = fma(p, m, Pair::both(-0.5f));
  Pair q = fma(Pair::both(GATE_Q4), m, Pair::both(GATE_Q3));
  q = fma(q, m, Pair::both(GATE_Q2));
  q = fma(q, m, Pair::both(GATE_Q1));
  const float2 d = fma(q, m, Pair::both(1.0f)).get(), x = mul(mul(m, m), Pair::both(-0.5f * LOG2_E)).get();
  p = mul(p, Pair::of(exp2_fast(x.x), exp2_fast(x.y)));
  p = mul(p, Pair::of(reciprocal_fast(d.x), reciprocal_fast(d.y)));
  return fma(m, p, Pair::of(positive_part(lo), positive_part(hi)));
}

template <int ACT>
__device__ __forceinline__ void activate_pair(float& lo, float& hi) {
  if constexpr (ACT == CCE_ACT_NONE || ACT == CCE_ACT_RELU) {
    lo = activate<ACT>(lo);
    hi = activate<ACT>(hi);
  } else {
    Pair y;
    if constexpr (ACT == CCE_ACT_GELU) {
      y = gelu_pair(lo, hi);
    } else {
      const Pair z = Pair::of(from_below(lo), from_below(hi));
      if constexpr (ACT == CCE_ACT_SILU) {
        y = mul(z, logistic_of_power(mul(z, Pair::both(-LOG2_E))));
      } else {
        y = mul(z, logistic_of_power(
                       mul(z, fma(mul(z, z), Pair::both(-2.0f * LOG2_E * GELU_C3), Pair::both(-2.0f * LOG2_E * GELU_C)))));
      }
    }
    const float2 f = y.get();
    lo = f.x;
    hi = f.y;
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

// AdamW over many tensors in one launch, states in 32 or 8 bits (include/cce_optim.h).
//
// Bound by memory: each value is read once and written once (bf16 parameters and
// gradients: 22 bytes a value with 32-bit states, 10 with 8-bit ones).  The tensors
// are cut into chunks, which the blocks of a launch take in turn; the table of
// tensors travels in the kernel's parameters (nothing to copy, nothing to keep alive
// for a captured graph).  The clipping factor is applied on the way, so the
// gradients need no pass of their own once their norm is known.
//
// 8 bits: a warp has a block of 256 values in its registers, eight a lane, so the
// new scales are two warp maxima and nothing is read twice.  What it spends is
// instructions, 66 a value, so the arithmetic is in packed fp32 pairs and the
// rounding to 8 bits in integers where it can be (136 M bf16 values, one gradient again
// and again from states of zero: 350 us for 381; in a training step's states 335).
//
// m and v are the sums of the formula with every operation rounded, no product fused
// into a sum: what decides over a value's rounding to 8 bits is then the same wherever
// the formula is evaluated in fp32.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/cce_optim.h"
#include "elements.cuh"
#include "internal.h"

namespace cce {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int VEC = 8;                // values of a thread at a time, in 32 bits as two vectors
constexpr int ROUND = THREADS * VEC;  // of a block
constexpr int BLOCKS_PER_SM = 4;
constexpr int MAX_TENSORS = 360;  // per launch: what 32 KB of parameters hold
constexpr int FEW_TENSORS = 16;  // in 1.5 KB: 16 tensors take 2.4 us and a call 10.3, with the table for all 2.8 and 11.8
constexpr int64_t MAX_ELEMENTS = int64_t(1) << 35;  // of one tensor
constexpr float E4M3_MAX = 448.0f, E4M3_MIN = 0x1p-9f, E4M3_NORMAL = 0x1p-6f, BLOCK_MIN = 0x1p-116f;
static_assert(CCE_ADAMW_BLOCK == 32 * VEC, "a block is a warp's");

struct Tensor {
  const void* g;
  void* p;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* rs;
  int64_t n;
  int64_t first_block;  // 8 bits: blocks of the call's tensors before this one
  uint32_t first_chunk;
  float decay;  // weight decay
  int wide;     // whole vectors start on their size
};

template <int M>
struct Batch {
  Tensor t[M];
  int count;
  int chunk;  // elements
  uint32_t chunks;
};

struct Rule {
  float beta1, rest1, beta2, rest2;  // rest: 1 - beta
  float eps;                         // times scale
  float scale;                       // a power of two on both sides of the quotient, so that a divisor is no subnormal
  float log1, log2;                  // natural logarithms of the betas
  float lr;
  float correct1, correct2;  // 1 - beta^t
  const int64_t* step;       // may be null
  const float* lr_ptr;       // may be null
  const float* norm;         // may be null
  float max_norm, eps_norm;
  uint32_t seed, t;
  float one;  // 1
};
static_assert(sizeof(Batch<MAX_TENSORS>) + sizeof(Rule) <= 32764, "kernel parameters");

template <int M>
__device__ __forceinline__ int find_tensor(const Batch<M>& b, uint32_t chunk) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.t[mid].first_chunk <= chunk) {
      lo = mid;
    } else {
      hi = mid - 1;
    }
  }
  return lo;
}

// The finaliser of MurmurHash3, without its first step.
__device__ __forceinline__ uint32_t mix_rest(uint32_t x) {
  x *= 0x85ebca6bu;
  x ^= x >> 13;
  x *= 0xc2b2ae35u;
  return x ^ x >> 16;
}
__device__ __forceinline__ uint32_t mix(uint32_t x) { return mix_rest(x ^ x >> 16); }

// What an update needs beside its values; the same in all threads.
struct Now {
  float factor;    // of the gradients
  float lr;
  float size;      // lr / (1 - beta1^t), times scale
  float inv_root;  // 1 / sqrt(1 - beta2^t), times scale
  uint32_t key;
};

__device__ __forceinline__ Now now_of(const Rule& r) {
  Now n;
  n.factor = 1.0f;
  if (r.norm) {  // as clipping does: NaN for a NaN norm, 1 where the quotient of infinities or zeros would be NaN
    const float norm = *r.norm, f = __frcp_rn(norm + r.eps_norm) * r.max_norm;
    n.factor = f < 1.0f || norm != norm ? f : 1.0f;
  }
  n.lr = r.lr_ptr ? *r.lr_ptr : r.lr;
  float c1 = r.correct1, c2 = r.correct2;
  uint32_t t = r.t;
  if (r.step) {
    const int64_t step = max(*r.step, static_cast<int64_t>(1));
    t = static_cast<uint32_t>(step);
    c1 = -expm1f(static_cast<float>(step) * r.log1);
    c2 = -expm1f(static_cast<float>(step) * r.log2);
  }
  n.size = n.lr / c1 * r.scale;
  n.inv_root = 1.0f / sqrtf(c2) * r.scale;
  n.key = mix(mix(r.seed) ^ t);
  return n;
}

// Two gradients' m and v.  The sums are fma(a, 1, b) with a 1 that the compiler does not know: it fuses a packed
// product into a packed addition, both rounded, all the same.
__device__ __forceinline__ void average(const Rule& r, const Now& now, Pair g, Pair& m, Pair& v) {
  const Pair one = Pair::both(r.one);
  g = mul(g, Pair::both(now.factor));
  m = fma(mul(Pair::both(r.beta1), m), one, mul(Pair::both(r.rest1), g));
  v = fma(mul(Pair::both(r.beta2), v), one, mul(mul(Pair::both(r.rest2), g), g));
}

// Two new weights.  (A divisor's root is 0 or at least 2^-75, that of fp32's least value, and eps is normal by its scale: the
// reciprocal, which takes subnormals for 0, sees none.  0 by 0, with eps = 0, is NaN.)
__device__ __forceinline__ Pair step_weights(const Rule& r, const Now& now, float keep, Pair w, Pair m, Pair root) {
  const float2 by = fma(root, Pair::both(now.inv_root), Pair::both(r.eps)).get();
  float lo, hi;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(lo) : "f"(by.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"(by.y));
  return fma(w, Pair::both(keep), mul(mul(Pair::both(-now.size), m), Pair::of(lo, hi)));
}

// U vectors of N values from element i on, THREADS vectors apart; all are loaded first.  (With vectors of four, each access
// of a warp to fp32 values is to whole sectors: eight took 504 us for 136 M bf16 values, 650 with masters, and two times
// four take 466 and 601.)
template <int N, int U, typename P, typename G, bool MASTER>
__device__ __forceinline__ void update_vectors(const Rule& r, const Now& now, float keep, const Tensor& t, int64_t i) {
  constexpr int APART = THREADS * N;
  Vec<G, N> g[U];
  Vec<P, N> p[U];
  Vec<float, N> w[U], m[U], v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = i + u * APART;
    g[u].load(static_cast<const G*>(t.g) + at);
    if constexpr (MASTER) {
      w[u].load(t.master + at);
    } else {
      p[u].load(static_cast<const P*>(t.p) + at);
    }
    m[u].load(static_cast<const float*>(t.m) + at);
    v[u].load(static_cast<const float*>(t.v) + at);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = i + u * APART;
    float wf[N], mf[N], vf[N];
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      constexpr int NEXT = N > 1 ? 1 : 0;
      const auto two = [&](const auto& x) { return Pair::of(x[u].get(e), x[u].get(e + NEXT)); };
      Pair m2 = two(m), v2 = two(v), w2;
      average(r, now, two(g), m2, v2);
      const float2 mm = m2.get(), vv = v2.get();
      if constexpr (MASTER) {
        w2 = two(w);
      } else {
        w2 = two(p);
      }
      const float2 ww = step_weights(r, now, keep, w2, m2, Pair::of(sqrtf(vv.x), sqrtf(vv.y))).get();
      wf[e] = ww.x, mf[e] = mm.x, vf[e] = vv.x;
      if constexpr (N > 1) wf[e + 1] = ww.y, mf[e + 1] = mm.y, vf[e + 1] = vv.y;
    }
    m[u].set(mf);
    v[u].set(vf);
    p[u].set(wf);
    m[u].store(static_cast<float*>(t.m) + at);
    v[u].store(static_cast<float*>(t.v) + at);
    p[u].store(static_cast<P*>(t.p) + at);
    if constexpr (MASTER) {
      w[u].set(wf);
      w[u].store(t.master + at);
    }
  }
}

template <int M, typename P, typename G, bool MASTER>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM) adamw_kernel(const __grid_constant__ Batch<M> b,
                                                                       const __grid_constant__ Rule r) {
  let_next_start();
  wait_for_previous();
  const Now now = now_of(r);
  for (uint32_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, c)];
    const int64_t at = static_cast<int64_t>(c - t.first_chunk) * b.chunk;
    const int64_t end = min(at + b.chunk, t.n);
    const float keep = 1.0f - now.lr * t.decay;
    int64_t from = at;
    if (t.wide) {
      constexpr int N = VEC / 2;
      const int64_t whole = at + (end - at) / N * N;
      int64_t i = at + threadIdx.x * N;
      for (; i + N * THREADS < whole; i += ROUND) update_vectors<N, 2, P, G, MASTER>(r, now, keep, t, i);
      if (i < whole) update_vectors<N, 1, P, G, MASTER>(r, now, keep, t, i);
      from = whole;
    }
    for (int64_t i = from + threadIdx.x; i < end; i += THREADS) update_vectors<1, 1, P, G, MASTER>(r, now, keep, t, i);
  }
}

// -------------------------------------------------------------------- 8 bits
__device__ __forceinline__ float2 from_e4m3(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Values that e4m3 holds (or NaN).
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Larger of two values; NaN wins.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_larger(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = larger(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The larger of `most` and two magnitudes; NaN wins.
__device__ __forceinline__ float largest(float most, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(most), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float smallest(float least, float a, float b) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(least), "f"(a), "f"(b));
  return r;
}

// 2^23 + the low (HIGH: the high) 16 bits of a word.
template <bool HIGH>
__device__ __forceinline__ float behind_2_23(uint32_t w) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, HIGH ? 0x7432 : 0x7410));
}

// Two a in [0, 448] to floor(a / step + u / 2^16) step; NaN stays NaN.  step: 2^-3 of a's power of two, 2^-9 at least; u:
// 16 random bits, given as 2^23 + u.  All but one rounding is of what is exact: a + u 2^-16 step as
// the formula rounds a / step + u 2^-16; the floor is a sum with 2^23 steps rounded down.  An a that roundings brought above
// 448, by 2^-22 of it at most, becomes 448 all the same: a / step is then below 14 + 2^-18.
__device__ __forceinline__ Pair round_e4m3(float a_lo, float a_hi, float u_lo, float u_hi) {
  constexpr uint32_t POWER = 0x7f800000u, LEAST = 121u << 23;  // 2^-6
  const Pair p = Pair::of(__uint_as_float(max(__float_as_uint(a_lo) & POWER, LEAST)),
                          __uint_as_float(max(__float_as_uint(a_hi) & POWER, LEAST)));  // 8 steps
  const Pair u = fma(Pair::of(u_lo, u_hi), Pair::both(0x1p-19f), Pair::both(-16.0f));
  const Pair s = fma(u, p, Pair::of(a_lo, a_hi));
  return fma(p, Pair::both(-0x1p20f), fma_down(p, Pair::both(0x1p20f), s));
}

// The same for an a in [2^-6, 448], as an e4m3 code in the top byte: fp32's exponent less 120 and three bits of its
// fraction, after u has been added to the twenty bits below them.  u: the low (HIGH: the high) 16 bits of `word`.
template <bool HIGH>
__device__ __forceinline__ uint32_t code_e4m3(float a, uint32_t word) {
  return __float_as_uint(a) * 16u + __byte_perm(word, 0x40u, HIGH ? 0x4325 : 0x4105);
}
__device__ __forceinline__ uint32_t top_bytes(const uint32_t* t) {
  return __byte_perm(__byte_perm(t[0], t[1], 0x73), __byte_perm(t[2], t[3], 0x73), 0x5410);
}

// The n values (n <= 256) of one block from element `at` of t on, by a warp.
template <typename P, typename G, bool MASTER>
__device__ __forceinline__ void update_block(const Rule& r, const Now& now, float keep, const Tensor& t, int64_t at,
                                             int n) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int64_t block = at / CCE_ADAMW_BLOCK, i = at + lane * VEC;
  const int mine = min(max(n - lane * VEC, 0), VEC);
  const bool wide = t.wide && mine == VEC;
  Vec<G, VEC> g;
  Vec<P, VEC> p;
  Vec<float, VEC> w;
  uint32_t mq[2] = {0u, 0u}, rq[2] = {0u, 0u};
  uint8_t* const m8 = static_cast<uint8_t*>(t.m) + i;
  uint8_t* const r8 = static_cast<uint8_t*>(t.v) + i;
  if (wide) {
    g.load(static_cast<const G*>(t.g) + i);
    if constexpr (MASTER) {
      w.load(t.master + i);
    } else {
      p.load(static_cast<const P*>(t.p) + i);
    }
    const uint2 a = *reinterpret_cast<const uint2*>(m8), b = *reinterpret_cast<const uint2*>(r8);
    mq[0] = a.x, mq[1] = a.y, rq[0] = b.x, rq[1] = b.y;
  } else {
    g.load_some(static_cast<const G*>(t.g) + i, 0, mine);
    if constexpr (MASTER) {
      w.load_some(t.master + i, 0, mine);
    } else {
      p.load_some(static_cast<const P*>(t.p) + i, 0, mine);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (e < mine) {
        mq[e / 4] |= static_cast<uint32_t>(m8[e]) << (8 * (e & 3));
        rq[e / 4] |= static_cast<uint32_t>(r8[e]) << (8 * (e & 3));
      }
    }
  }
  const Pair ms = Pair::both(t.ms[block]), rs = Pair::both(t.rs[block]);
  Pair m2[VEC / 2], r2[VEC / 2];
  float wf[VEC], m_most = 0.0f, r_most = 0.0f;
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    const float2 a = from_e4m3(mq[e / 4] >> (8 * (e & 3))), b = from_e4m3(rq[e / 4] >> (8 * (e & 3)));
    Pair m = mul(Pair::of(a.x, a.y), ms), v = mul(Pair::of(b.x, b.y), rs);
    v = mul(v, v);
    average(r, now, Pair::of(g.get(e), g.get(e + 1)), m, v);
    const float2 mm = m.get(), vv = v.get();
    const float root[2] = {__fsqrt_rn(vv.x), __fsqrt_rn(vv.y)};
    m2[e / 2] = m;
    r2[e / 2] = Pair::of(root[0], root[1]);
    Pair w2;
    if constexpr (MASTER) {
      w2 = Pair::of(w.get(e), w.get(e + 1));
    } else {
      w2 = Pair::of(p.get(e), p.get(e + 1));
    }
    const float2 ww = step_weights(r, now, keep, w2, m, r2[e / 2]).get();
    wf[e] = ww.x, wf[e + 1] = ww.y;
    // (elements behind the tensor's end are zeros, and so are their states)
    m_most = largest(m_most, mm.x, mm.y);
    r_most = largest(r_most, root[0], root[1]);
  }
  m_most = warp_larger(m_most);
  r_most = warp_larger(r_most);
  const bool m_none = m_most < BLOCK_MIN, r_none = r_most < BLOCK_MIN;
  const float m_inv = m_none ? 0.0f : __frcp_rn(m_most) * E4M3_MAX, r_inv = r_none ? 0.0f : __frcp_rn(r_most) * E4M3_MAX;
  const uint64_t place = static_cast<uint64_t>(t.first_block + block) * CCE_ADAMW_BLOCK + lane * VEC;
  const uint32_t key = mix(now.key ^ static_cast<uint32_t>(place >> 32));
  // mix(place + e ^ key) for the lane's e: place is a multiple of 8, so that the first shift is the same for all
  const uint32_t start = static_cast<uint32_t>(place) ^ key, shifted = start ^ start >> 16;
  uint32_t word[VEC], mw[2], rw[2];
  float ma[VEC], ra[VEC], least = E4M3_MAX;
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    word[e] = mix_rest(shifted ^ e), word[e + 1] = mix_rest(shifted ^ (e + 1));
    const float2 a = mul(m2[e / 2], Pair::both(m_inv)).get(), b = mul(r2[e / 2], Pair::both(r_inv)).get();
    ma[e] = a.x, ma[e + 1] = a.y, ra[e] = b.x, ra[e + 1] = b.y;
    least = smallest(smallest(least, fabsf(a.x), fabsf(a.y)), b.x, b.y);
  }
  if (least >= E4M3_NORMAL) {
    uint32_t mt[VEC], rt[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      mt[e] = (code_e4m3<false>(ma[e], word[e]) & 0x7fffffffu) | (__float_as_uint(ma[e]) & 0x80000000u);
      rt[e] = code_e4m3<true>(ra[e], word[e]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) mw[h] = top_bytes(mt + 4 * h), rw[h] = top_bytes(rt + 4 * h);
  } else {
    float mo[VEC], ro[VEC];
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const uint32_t x = word[e], y = word[e + 1];
      const float2 mr = round_e4m3(fabsf(ma[e]), fabsf(ma[e + 1]), behind_2_23<false>(x), behind_2_23<false>(y)).get();
      const float2 rr = round_e4m3(ra[e], ra[e + 1], behind_2_23<true>(x), behind_2_23<true>(y)).get();
      mo[e] = copysignf(mr.x, ma[e]), mo[e + 1] = copysignf(mr.y, ma[e + 1]);
      // a positive root stays one (magnitudes compare as their bits do, NaN above all)
      const auto positive = [](float q, float of) {
        return __uint_as_float(max(__float_as_uint(q), min(__float_as_uint(of), 1u) * __float_as_uint(E4M3_MIN)));
      };
      ro[e] = positive(rr.x, ra[e]), ro[e + 1] = positive(rr.y, ra[e + 1]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mw[h] = to_e4m3(mo[4 * h], mo[4 * h + 1]) | to_e4m3(mo[4 * h + 2], mo[4 * h + 3]) << 16;
      rw[h] = to_e4m3(ro[4 * h], ro[4 * h + 1]) | to_e4m3(ro[4 * h + 2], ro[4 * h + 3]) << 16;
    }
  }
  p.set(wf);
  if constexpr (MASTER) w.set(wf);
  if (wide) {
    p.store(static_cast<P*>(t.p) + i);
    if constexpr (MASTER) w.store(t.master + i);
    *reinterpret_cast<uint2*>(m8) = make_uint2(mw[0], mw[1]);
    *reinterpret_cast<uint2*>(r8) = make_uint2(rw[0], rw[1]);
  } else {
    p.store_some(static_cast<P*>(t.p) + i, 0, mine);
    if constexpr (MASTER) w.store_some(t.master + i, 0, mine);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (e < mine) {
        m8[e] = static_cast<uint8_t>(mw[e / 4] >> (8 * (e & 3)));
        r8[e] = static_cast<uint8_t>(rw[e / 4] >> (8 * (e & 3)));
      }
    }
  }
  if (lane == 0) {
    t.ms[block] = m_none ? 0.0f : m_most * (1.0f / E4M3_MAX);
    t.rs[block] = r_none ? 0.0f : r_most * (1.0f / E4M3_MAX);
  }
}

template <int M, typename P, typename G, bool MASTER>
__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM) adamw8_kernel(const __grid_constant__ Batch<M> b,
                                                                        const __grid_constant__ Rule r) {
  let_next_start();
  wait_for_previous();
  const Now now = now_of(r);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  for (uint32_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, c)];
    const int64_t at = static_cast<int64_t>(c - t.first_chunk) * b.chunk;
    const int64_t end = min(at + b.chunk, t.n);
    const float keep = 1.0f - now.lr * t.decay;
    for (int64_t i = at + warp * CCE_ADAMW_BLOCK; i < end; i += WARPS * CCE_ADAMW_BLOCK)
      update_block<P, G, MASTER>(r, now, keep, t, i, static_cast<int>(min(end - i, static_cast<int64_t>(CCE_ADAMW_BLOCK))));
  }
}

// ---------------------------------------------------------------------- host
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t type_bytes(int t) { return t == CCE_F32 ? 4 : 2; }
bool type_ok(int t) { return t == CCE_F32 || t == CCE_F16 || t == CCE_BF16; }
bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }
bool finite_positive(double v) { return std::isfinite(v) && v >= 0.0; }

cce_status check_tensor(const cce_adamw_tensor& t, bool eight) {
  if (!type_ok(t.grad_type) || !type_ok(t.param_type) || !finite_positive(t.weight_decay)) return CCE_ERR_ARG;
  if (t.n < 0 || t.n >= MAX_ELEMENTS) return CCE_ERR_SHAPE;
  if (t.n == 0) return CCE_OK;
  if (!t.grad || !t.param || !t.exp_avg || !t.exp_avg_sq || (eight && (!t.exp_avg_scale || !t.rms_scale)))
    return CCE_ERR_NULL;
  if (!multiple(t.grad, type_bytes(t.grad_type)) || !multiple(t.param, type_bytes(t.param_type)) ||
      !multiple(t.master, 4) || (!eight && (!multiple(t.exp_avg, 4) || !multiple(t.exp_avg_sq, 4))) ||
      (eight && (!multiple(t.exp_avg_scale, 4) || !multiple(t.rms_scale, 4))))
    return CCE_ERR_ALIGN;
  return CCE_OK;
}

// Memory that is written and overlaps other memory would be read and written in
// any order by the blocks of a launch.
struct Span {
  uintptr_t lo, hi;
  bool out;
};

cce_status check_overlap(const cce_adamw_tensor* t, int64_t n, bool eight) {
  Span* spans = new (std::nothrow) Span[7 * static_cast<size_t>(std::max<int64_t>(1, n))];
  if (!spans) return CCE_ERR_CUDA;
  int64_t m = 0;
  const auto add = [&](const void* p, int64_t bytes, bool out) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (p) spans[m++] = Span{lo, lo + static_cast<uintptr_t>(bytes), out};
  };
  for (int64_t i = 0; i < n; ++i) {
    const cce_adamw_tensor& a = t[i];
    if (a.n == 0) continue;
    add(a.grad, a.n * type_bytes(a.grad_type), false);
    add(a.param, a.n * type_bytes(a.param_type), true);
    add(a.master, a.n * 4, true);
    add(a.exp_avg, a.n * (eight ? 1 : 4), true);
    add(a.exp_avg_sq, a.n * (eight ? 1 : 4), true);
    if (eight) {
      add(a.exp_avg_scale, cdiv(a.n, CCE_ADAMW_BLOCK) * 4, true);
      add(a.rms_scale, cdiv(a.n, CCE_ADAMW_BLOCK) * 4, true);
    }
  }
  std::sort(spans, spans + m, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t end_any = 0, end_out = 0;
  bool bad = false;
  for (int64_t i = 0; i < m; ++i) {
    bad = bad || spans[i].lo < (spans[i].out ? end_any : end_out);
    end_any = std::max(end_any, spans[i].hi);
    if (spans[i].out) end_out = std::max(end_out, spans[i].hi);
  }
  delete[] spans;
  return bad ? CCE_ERR_ARG : CCE_OK;
}

struct Call {
  const cce_adamw_tensor* t;
  int64_t n;
  bool eight;
  int chunk, grid;
  Rule r;
  cudaStream_t s;
  int launches;
};

template <int M, typename P, typename G, bool MASTER>
cudaError_t run_batches(Call& c) {
  Batch<M> b;
  int64_t next = 0, blocks = 0;
  while (next < c.n) {
    b.count = 0;
    b.chunk = c.chunk;
    int64_t chunks = 0;
    for (; next < c.n && b.count < M; ++next) {
      const cce_adamw_tensor& a = c.t[next];
      const int64_t before = blocks;
      blocks += cdiv(a.n, CCE_ADAMW_BLOCK);
      if (a.n == 0 || a.param_type != ElemType<P>::id || a.grad_type != ElemType<G>::id || !a.master == MASTER)
        continue;
      Tensor& t = b.t[b.count++];
      t.g = a.grad;
      t.p = a.param;
      t.master = a.master;
      t.m = a.exp_avg;
      t.v = a.exp_avg_sq;
      t.ms = a.exp_avg_scale;
      t.rs = a.rms_scale;
      t.n = a.n;
      t.first_block = before;
      t.first_chunk = static_cast<uint32_t>(chunks);
      t.decay = a.weight_decay;
      t.wide = multiple(a.grad, 16) && multiple(a.param, 16) && multiple(a.master, 16) &&
               multiple(a.exp_avg, c.eight ? 8 : 16) && multiple(a.exp_avg_sq, c.eight ? 8 : 16);
      chunks += cdiv(a.n, c.chunk);
    }
    if (b.count == 0) continue;
    b.chunks = static_cast<uint32_t>(chunks);
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(c.grid, chunks)));
    const cudaError_t e = c.eight ? launch_after(adamw8_kernel<M, P, G, MASTER>, grid, dim3(THREADS), 0, 1, c.s, b, c.r)
                                  : launch_after(adamw_kernel<M, P, G, MASTER>, grid, dim3(THREADS), 0, 1, c.s, b, c.r);
    if (e != cudaSuccess) return e;
    ++c.launches;
  }
  return cudaSuccess;
}

template <typename P, typename G, bool MASTER>
cudaError_t run_kind(Call& c) {
  return c.n <= FEW_TENSORS ? run_batches<FEW_TENSORS, P, G, MASTER>(c) : run_batches<MAX_TENSORS, P, G, MASTER>(c);
}

template <typename P, bool MASTER>
cudaError_t run_param(Call& c, int grad_type) {
  if (grad_type == CCE_F32) return run_kind<P, float, MASTER>(c);
  return grad_type == CCE_BF16 ? run_kind<P, __nv_bfloat16, MASTER>(c) : run_kind<P, __half, MASTER>(c);
}

cudaError_t run_all(Call& c) {
  // one launch for each kind of types that there is
  bool seen[3][3][2] = {};
  for (int64_t i = 0; i < c.n; ++i) {
    const cce_adamw_tensor& a = c.t[i];
    if (a.n == 0) continue;
    bool& done = seen[a.param_type][a.grad_type][a.master != nullptr];
    if (done) continue;
    done = true;
    cudaError_t e;
    if (a.param_type == CCE_F32) {
      e = a.master ? run_param<float, true>(c, a.grad_type) : run_param<float, false>(c, a.grad_type);
    } else if (a.param_type == CCE_BF16) {
      e = a.master ? run_param<__nv_bfloat16, true>(c, a.grad_type) : run_param<__nv_bfloat16, false>(c, a.grad_type);
    } else {
      e = a.master ? run_param<__half, true>(c, a.grad_type) : run_param<__half, false>(c, a.grad_type);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace cce

using namespace cce;

extern "C" {

int cce_optim_abi_version(void) { return 100; }

cce_status cce_adamw_step(const cce_adamw_tensor* tensors, int64_t n_tensors, int state_bits,
                          const cce_adamw_options* o, void* stream) {
  if (n_tensors < 0) return CCE_ERR_SHAPE;
  if (!o || (n_tensors > 0 && !tensors)) return CCE_ERR_NULL;
  const auto beta_ok = [](double b) { return b >= 0.0 && b < 1.0; };
  if ((state_bits != 32 && state_bits != 8) || !beta_ok(o->beta1) || !beta_ok(o->beta2) || !finite_positive(o->lr) ||
      !finite_positive(o->eps) || (!o->step_ptr && o->step < 1))
    return CCE_ERR_ARG;
  if (o->norm && (!(o->max_norm >= 0.0f) || !finite_positive(o->eps_norm))) return CCE_ERR_ARG;
  if (!multiple(o->step_ptr, 8) || !multiple(o->lr_ptr, 4) || !multiple(o->norm, 4)) return CCE_ERR_ALIGN;
  const bool eight = state_bits == 8;
  int64_t total = 0;
  for (int64_t i = 0; i < n_tensors; ++i) {
    const cce_status st = check_tensor(tensors[i], eight);
    if (st != CCE_OK) return st;
    total += tensors[i].n;
  }
  cce_status st = check_overlap(tensors, n_tensors, eight);
  if (st != CCE_OK) return st;
  int sms = 0;
  st = static_cast<cce_status>(device_ready(&sms));
  if (st != CCE_OK) return st;
  const double t = static_cast<double>(o->step);
  Rule r{};
  r.beta1 = static_cast<float>(o->beta1);
  r.rest1 = static_cast<float>(1.0 - o->beta1);
  r.beta2 = static_cast<float>(o->beta2);
  r.rest2 = static_cast<float>(1.0 - o->beta2);
  // an eps among fp32's subnormals, from 2^-150 on, becomes a normal value, and what stands beside it is scaled likewise
  r.scale = o->eps > 0.0 && o->eps < 0x1p-126 ? 0x1p24f : 1.0f;
  r.eps = static_cast<float>(o->eps * r.scale);
  r.log1 = static_cast<float>(std::log(o->beta1));
  r.log2 = static_cast<float>(std::log(o->beta2));
  r.lr = static_cast<float>(o->lr);
  r.correct1 = static_cast<float>(1.0 - std::pow(o->beta1, t));
  r.correct2 = static_cast<float>(1.0 - std::pow(o->beta2, t));
  r.step = o->step_ptr;
  r.lr_ptr = o->lr_ptr;
  r.norm = o->norm;
  r.max_norm = o->max_norm;
  r.eps_norm = o->eps_norm;
  r.seed = o->seed;
  r.t = static_cast<uint32_t>(o->step);
  r.one = 1.0f;
  // four rounds of a block, one where that leaves blocks without work
  const int grid = sms * BLOCKS_PER_SM;
  Call c{tensors, n_tensors, eight, total >= int64_t(4) * grid * ROUND ? 4 * ROUND : ROUND, grid, r,
         static_cast<cudaStream_t>(stream), 0};
  const cudaError_t e = run_all(c);
  count_launches(c.launches);
  return e == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

}  // extern "C"

// Layer norm and RMS norm kernels, forward and backward.
//
//   layer norm  m = sum x / D, r = 1 / sqrt(sum (x - m)^2 / D + eps), z = (x - m) r, y = z w + b
//   RMS norm    m = 0,         r = 1 / sqrt(sum x^2 / D + eps),       z = x r,       y = z (o + w)
//   backward    g = dy (o + w);  dx = r (g - sum(g) / D - z sum(g z) / D), the sum(g) term for layer norm only
//               dw = sum over rows of dy z;  db = sum over rows of dy
//
// All of it is bound by memory: a row is read once, held in registers as raw
// words, reduced, and written.  The variance is the sum of squared deviations
// from the mean, taken over the registers, so nothing cancels.
//
// A row belongs to a group of threadIdx.x = 0 .. tpr - 1 (tpr a power of two up
// to 32, or a multiple of 32); a block has blockDim.y groups.  Thread l of a
// group holds the vectors l, l + tpr, ..., K of them.
#pragma once

#include <algorithm>

#include "elements.cuh"
#include "norm.h"
#include "ptx.cuh"

namespace cce {
namespace norm {

constexpr int MAX_THREADS = 512;

__device__ __forceinline__ float lanes_sum(float v, int width) {
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Barrier over the warps of one group (the whole block when it is the only one).
__device__ __forceinline__ void group_sync() {
  if (blockDim.y == 1) {
    __syncthreads();
  } else {
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(blockDim.x) : "memory");
  }
}

// Sum over the group; sm has one slot for each of the group's warps.
__device__ __forceinline__ float group_sum(float v, float* sm) {
  const int tpr = blockDim.x;
  if (tpr <= 32) return lanes_sum(v, tpr);
  v = lanes_sum(v, 32);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  group_sync();
  float t = 0.0f;
  for (int i = 0; i < tpr >> 5; ++i) t += sm[i];
  return t;
}

// Of two values; without BOTH, of .y alone.
template <bool BOTH>
__device__ __forceinline__ float2 group_sum2(float2 v, float2* sm) {
  const int tpr = blockDim.x;
  const int width = tpr < 32 ? tpr : 32;
  if (BOTH) v.x = lanes_sum(v.x, width);
  v.y = lanes_sum(v.y, width);
  if (tpr <= 32) return v;
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  group_sync();
  float2 t = make_float2(0.0f, 0.0f);
  for (int i = 0; i < tpr >> 5; ++i) {
    if (BOTH) t.x += sm[i].x;
    t.y += sm[i].y;
  }
  return t;
}

template <bool LAYER, int VEC>
__device__ __forceinline__ void load_gain(const void* w, int p_type, float offset, int64_t c, float (&g)[VEC]) {
  if (w) {
    load_param<VEC>(w, p_type, c, g);
    if (!LAYER) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) g[e] += offset;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = 1.0f;
  }
}

template <bool LAYER, int VEC>
__device__ __forceinline__ void load_bias(const void* b, int p_type, int64_t c, float (&f)[VEC]) {
  if (LAYER && b) {
    load_param<VEC>(b, p_type, c, f);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = 0.0f;
  }
}

// Pair i of the K * VEC / 2 fp32 pairs in the K vectors of a thread.  With VEC = 1
// a pair is two of the thread's columns.
template <typename T, int VEC, int K>
__device__ __forceinline__ Pair pair_of(const Vec<T, VEC> (&v)[K], int i) {
  return Pair::of(v[2 * i / VEC].get(2 * i % VEC), v[(2 * i + 1) / VEC].get((2 * i + 1) % VEC));
}

// Whether a thread holds its vector k.  Every thread holds the first KF, so
// that only the others are checked.
template <int KF>
__device__ __forceinline__ bool holds(int k, int vecs) {
  return k < KF || static_cast<int>(threadIdx.x + k * blockDim.x) < vecs;
}

// Parameters in shared memory as fp32.  The vectors' float4 quarters lie apart,
// so that a warp's 16-byte reads fall on consecutive addresses.
template <int VEC>
__device__ __forceinline__ void put_param(float* sm, int vecs, int c, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    sm[c] = f[0];
  } else {
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h)
      reinterpret_cast<float4*>(sm)[h * vecs + c] = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
  }
}

template <int VEC>
__device__ __forceinline__ void get_param(const float* sm, int vecs, int c, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = sm[c];
  } else {
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) {
      const float4 v = reinterpret_cast<const float4*>(sm)[h * vecs + c];
      f[4 * h] = v.x;
      f[4 * h + 1] = v.y;
      f[4 * h + 2] = v.z;
      f[4 * h + 3] = v.w;
    }
  }
}

// ------------------------------------------------------------------ forward
// Few rows: a block of up to 512 threads per row, so that a row's loads are all
// in flight at once; parameters are loaded beside them.
template <typename TX, typename TY, int VEC, int K, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) fwd_few_kernel(NormFwd a) {
  __shared__ float sm[2][MAX_THREADS / 32];
  const int l = threadIdx.x, tpr = blockDim.x;
  const int64_t n = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n));
  Vec<TX, VEC> xv[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (l + k * tpr) * VEC;
    xv[k].zero();
    if (c < a.D) xv[k].load(x + c);
  }
  float w[K][VEC], b[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (l + k * tpr) * VEC;
    if (c < a.D) {
      load_gain<LAYER, VEC>(a.w, a.p_type, a.offset, c, w[k]);
      load_bias<LAYER, VEC>(a.b, a.p_type, c, b[k]);
    }
  }
  const float fd = static_cast<float>(a.D);
  float mean = 0.0f;
  if (LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += xv[k].get(e);
    }
    mean = group_sum(s, sm[0]) / fd;
  }
  float q = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if ((l + k * tpr) * VEC < a.D) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = xv[k].get(e) - mean;
        q += d * d;
      }
    }
  }
  const float rstd = 1.0f / sqrtf(group_sum(q, sm[1]) / fd + a.eps);
  if (l == 0) {
    if (LAYER && a.mean) a.mean[n] = mean;
    if (a.rstd) a.rstd[n] = rstd;
  }
  TY* y = static_cast<TY*>(a.y) + n * a.D;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (l + k * tpr) * VEC;
    if (c < a.D) {
      float o[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = (xv[k].get(e) - mean) * rstd * w[k][e] + b[k][e];
      Vec<TY, VEC> out;
      out.set(o);
      out.store(y + c);
    }
  }
}

// Many rows: persistent blocks whose groups walk rows at a stride of all groups.
// A thread holds up to 64 values of a row, so that most rows are a warp's or
// less and their sums are shuffles alone; the next row is loaded while this one
// is reduced.  The parameters wait in shared memory as fp32.
template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) fwd_kernel(NormFwd a) {
  constexpr int E = K * VEC / 2;
  extern __shared__ __align__(16) float params[];  // gain [D], then the bias [D] of a layer norm
  __shared__ float sm[4][MAX_THREADS / 32];
  const int l = threadIdx.x, tpr = blockDim.x, groups = blockDim.y;
  const int vecs = a.D / VEC, slot = threadIdx.y * (tpr >> 5);
  float* gain = params;
  float* bias = params + a.D;
  const int step = gridDim.x * groups;
  Vec<TX, VEC> xv[K];
#pragma unroll
  for (int k = 0; k < K; ++k) xv[k].zero();
  auto load_row = [&](int64_t n) {
    if (n >= a.N) return;
    const TX* x = static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (holds<KF>(k, vecs)) xv[k].load(x + (l + k * tpr) * VEC);
    }
  };
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
  load_row(base + threadIdx.y);
  for (int c = threadIdx.y * tpr + l; c < vecs; c += tpr * groups) {
    float f[VEC];
    load_gain<LAYER, VEC>(a.w, a.p_type, a.offset, static_cast<int64_t>(c) * VEC, f);
    put_param<VEC>(gain, vecs, c, f);
    if (LAYER) {
      load_bias<LAYER, VEC>(a.b, a.p_type, static_cast<int64_t>(c) * VEC, f);
      put_param<VEC>(bias, vecs, c, f);
    }
  }
  __syncthreads();
  const float fd = static_cast<float>(a.D);
  int buf = 0;
  for (; base < a.N; base += step) {
    const int64_t n = base + threadIdx.y;
    Pair d[E];
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = pair_of<TX, VEC, K>(xv, i);
    load_row(n + step);
    float mean = 0.0f;
    if (LAYER) {
      Pair s[2] = {Pair::both(0.0f), Pair::both(0.0f)};  // two chains
#pragma unroll
      for (int i = 0; i < E; ++i) s[i & 1] = add(s[i & 1], d[i]);
      mean = group_sum(add(s[0], s[1]).sum(), sm[buf] + slot) / fd;
      const Pair minus = Pair::both(-mean);
#pragma unroll
      for (int i = 0; i < E; ++i) d[i] = add(d[i], minus);
    }
    Pair q[2] = {Pair::both(0.0f), Pair::both(0.0f)};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int k0 = 2 * i / VEC, k1 = (2 * i + 1) / VEC;
      if constexpr (LAYER && VEC == 1) {  // columns that are not there would add mean^2
        const float2 f = d[i].get();
        d[i] = Pair::of(holds<KF>(k0, vecs) ? f.x : 0.0f, holds<KF>(k1, vecs) ? f.y : 0.0f);
        q[i & 1] = fma(d[i], d[i], q[i & 1]);
      } else {
        if (!LAYER || holds<KF>(k0, vecs)) q[i & 1] = fma(d[i], d[i], q[i & 1]);
      }
    }
    const float rstd = 1.0f / sqrtf(group_sum(add(q[0], q[1]).sum(), sm[buf + 1] + slot) / fd + a.eps);
    buf ^= 2;  // the other slots for the next row: a slower warp may still read these
    if (n >= a.N) continue;
    if (l == 0) {
      if (LAYER && a.mean) a.mean[n] = mean;
      if (a.rstd) a.rstd[n] = rstd;
    }
    TY* y = static_cast<TY*>(a.y) + n * a.D;
    const Pair r = Pair::both(rstd);
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = mul(d[i], r);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (holds<KF>(k, vecs)) {
        const int c = l + k * tpr;
        float w[VEC], b[VEC], o[VEC];
        get_param<VEC>(gain, vecs, c, w);
        if (LAYER) get_param<VEC>(bias, vecs, c, b);
        if constexpr (VEC == 1) {
          const float2 f = d[k / 2].get();
          const float z = k & 1 ? f.y : f.x;
          o[0] = LAYER ? z * w[0] + b[0] : z * w[0];
        } else {
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) {
            const Pair z = d[k * VEC / 2 + i], g = Pair::of(w[2 * i], w[2 * i + 1]);
            const float2 f = (LAYER ? fma(z, g, Pair::of(b[2 * i], b[2 * i + 1])) : mul(z, g)).get();
            o[2 * i] = f.x;
            o[2 * i + 1] = f.y;
          }
        }
        Vec<TY, VEC> out;
        out.set(o);
        out.store(y + static_cast<int64_t>(c) * VEC);
      }
    }
  }
}

// Rows too long for the registers of one block: one block per row, which
// reads it once per sum and once more to write (from L2 after the first time).
template <typename TX, typename TY, int VEC, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) fwd_long_kernel(NormFwd a) {
  __shared__ float sm[2][MAX_THREADS / 32];
  const int64_t n = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n));
  const float fd = static_cast<float>(a.D);
  const int64_t first = static_cast<int64_t>(threadIdx.x) * VEC, step = static_cast<int64_t>(blockDim.x) * VEC;
  float mean = 0.0f;
  if (LAYER) {
    float s = 0.0f;
#pragma unroll 4
    for (int64_t c = first; c < a.D; c += step) {
      Vec<TX, VEC> v;
      v.load(x + c);
      float t = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) t += v.get(e);
      s += t;
    }
    mean = group_sum(s, sm[0]) / fd;
  }
  float q = 0.0f;
#pragma unroll 4
  for (int64_t c = first; c < a.D; c += step) {
    Vec<TX, VEC> v;
    v.load(x + c);
    float t = 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float d = v.get(e) - mean;
      t += d * d;
    }
    q += t;
  }
  const float rstd = 1.0f / sqrtf(group_sum(q, sm[1]) / fd + a.eps);
  if (threadIdx.x == 0) {
    if (LAYER && a.mean) a.mean[n] = mean;
    if (a.rstd) a.rstd[n] = rstd;
  }
  TY* y = static_cast<TY*>(a.y) + n * a.D;
#pragma unroll 2
  for (int64_t c = first; c < a.D; c += step) {
    Vec<TX, VEC> v;
    v.load(x + c);
    float w[VEC], b[VEC], o[VEC];
    load_gain<LAYER, VEC>(a.w, a.p_type, a.offset, c, w);
    load_bias<LAYER, VEC>(a.b, a.p_type, c, b);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = (v.get(e) - mean) * rstd * w[e] + b[e];
    Vec<TY, VEC> out;
    out.set(o);
    out.store(y + c);
  }
}

// ----------------------------------------------------------------- backward
// Persistent blocks, one per SM: a group walks rows at a stride of all groups,
// and each thread keeps the parameter gradients of its own columns in registers
// over all of them.  At the end a block adds its groups in order and writes one
// partial row; reduce_kernel adds the blocks in order.  Few rows are left to the
// blocks of one cluster, which add their sums themselves: no second launch.
//
// The columns' sums are what fills the registers, so a thread holds 16 values of
// a row (32 in rows that need it) and a row is spread over more threads than in
// the forward.  PREFETCH loads the next row while this one is reduced.
template <typename TX, int VEC, int K, bool LAYER>
constexpr int bwd_threads() {
  return !LAYER && sizeof(TX) == 2 && VEC > 1 && K * VEC <= 16 ? 768 : 512;
}

__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float f;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(addr) : "memory");
  return f;
}

template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER, bool PREFETCH>
__global__ void __launch_bounds__(bwd_threads<TX, VEC, K, LAYER>(), 1) bwd_kernel(NormBwd a) {
  constexpr int E = K * VEC / 2;
  extern __shared__ __align__(16) float shared[];  // the gain [D]; at the end the groups' sums
  __shared__ float2 sm[2][bwd_threads<TX, VEC, K, LAYER>() / 32];
  const int l = threadIdx.x, tpr = blockDim.x, groups = blockDim.y;
  const int vecs = a.D / VEC, slot = threadIdx.y * (tpr >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_d = 1.0f / static_cast<float>(a.D);

  Vec<TX, VEC> xv[K];
  Vec<TY, VEC> gv[K];
  float mean = 0.0f, rstd = 0.0f;
  auto load_row = [&](int64_t n) {
    if (n < a.N) {
      const TX* x = static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n));
      const TY* dy = static_cast<const TY*>(a.dy) + a.gm.at(static_cast<int>(n));
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (holds<KF>(k, vecs)) {
          xv[k].load(x + (l + k * tpr) * VEC);
          gv[k].load(dy + (l + k * tpr) * VEC);
        }
      }
      if (LAYER) mean = a.mean[n];
      rstd = a.rstd[n];
    } else {  // a row of zeros adds nothing
#pragma unroll
      for (int k = 0; k < K; ++k) gv[k].zero();
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    xv[k].zero();
    gv[k].zero();
  }
  let_next_start();
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
  if (PREFETCH) load_row(base + threadIdx.y);
  for (int c = threadIdx.y * tpr + l; c < vecs; c += tpr * groups) {
    float f[VEC];
    load_gain<LAYER, VEC>(a.w, a.p_type, a.offset, static_cast<int64_t>(c) * VEC, f);
    put_param<VEC>(shared, vecs, c, f);
  }
  __syncthreads();

  Pair aw[E], ab[LAYER ? E : 1];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    aw[i] = Pair::both(0.0f);
    if (LAYER) ab[i] = Pair::both(0.0f);
  }
  int buf = 0;
  for (; base < a.N; base += step) {
    const int64_t n = base + threadIdx.y;
    if (!PREFETCH) load_row(n);
    Vec<TX, VEC> x[K];
    Vec<TY, VEC> g[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = xv[k];
      g[k] = gv[k];
    }
    const float row_rstd = rstd, row_mean = mean;
    if (PREFETCH) load_row(n + step);
    // z = x rstd - mean rstd
    const Pair r = Pair::both(row_rstd), m = Pair::both(-row_mean * row_rstd);
    float2 s;
    {
      Pair s1 = Pair::both(0.0f), s2 = Pair::both(0.0f);
      auto gather = [&](int i, Pair w) {
        const Pair xp = pair_of<TX, VEC, K>(x, i), dp = pair_of<TY, VEC, K>(g, i);
        const Pair z = LAYER ? fma(xp, r, m) : mul(xp, r);
        const Pair t = mul(dp, w);
        aw[i] = fma(dp, z, aw[i]);
        if (LAYER) {
          ab[i] = add(ab[i], dp);
          s1 = add(s1, t);
        }
        s2 = fma(t, z, s2);
      };
      if constexpr (VEC == 1) {
#pragma unroll
        for (int k = 0; k < K; k += 2) {  // where a column is not there its dy is 0, and any gain does
          gather(k / 2, Pair::of(shared[holds<KF>(k, vecs) ? l + k * tpr : 0],
                                 shared[holds<KF>(k + 1, vecs) ? l + (k + 1) * tpr : 0]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!holds<KF>(k, vecs)) continue;
          float w[VEC];
          get_param<VEC>(shared, vecs, l + k * tpr, w);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) gather(k * VEC / 2 + i, Pair::of(w[2 * i], w[2 * i + 1]));
        }
      }
      s = make_float2(LAYER ? s1.sum() : 0.0f, s2.sum());
    }
    if (!a.dx) continue;
    s = group_sum2<LAYER>(s, sm[buf] + slot);
    buf ^= 1;  // the other slots for the next row: a slower warp may still read these
    if (n >= a.N) continue;
    TX* dx = static_cast<TX*>(a.dx) + n * a.D;
    const Pair c1 = Pair::both(-s.x * inv_d * row_rstd), c2 = Pair::both(-s.y * inv_d * row_rstd);
    // rstd (g - sum(g) / D - z sum(g z) / D)
    auto grad = [&](int i, Pair w) {
      const Pair xp = pair_of<TX, VEC, K>(x, i), dp = pair_of<TY, VEC, K>(g, i);
      const Pair z = LAYER ? fma(xp, r, m) : mul(xp, r);
      return fma(mul(dp, w), r, LAYER ? fma(z, c2, c1) : mul(z, c2)).get();
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!holds<KF>(k, vecs)) continue;
      float w[VEC], f[VEC];
      get_param<VEC>(shared, vecs, l + k * tpr, w);
      if constexpr (VEC == 1) {
        const float2 t = grad(k / 2, Pair::both(w[0]));
        f[0] = k & 1 ? t.y : t.x;
      } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 t = grad(k * VEC / 2 + i, Pair::of(w[2 * i], w[2 * i + 1]));
          f[2 * i] = t.x;
          f[2 * i + 1] = t.y;
        }
      }
      Vec<TX, VEC> out;
      out.set(f);
      out.store(dx + (l + k * tpr) * VEC);
    }
  }

  // Several groups: their sums side by side in shared memory (the weight's, then
  // the bias's), added in order.  One group: straight into the partial row.
  if (!a.dw && !a.db) return;
  const bool side_by_side = groups > 1 || a.cluster;
  if (side_by_side) __syncthreads();  // the gain has been read
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.D;
#pragma unroll
  for (int pass = 0; pass < (LAYER ? 2 : 1); ++pass) {
    if (!(pass == 0 ? a.dw : a.db)) continue;
    float* part =
        side_by_side ? shared + (pass * groups + threadIdx.y) * a.D : (pass == 0 ? a.part_w : a.part_b) + row;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!holds<KF>(k, vecs)) continue;
      float* to = part + (l + k * tpr) * VEC;
      if constexpr (VEC == 1) {
        const float2 t = (pass == 0 ? aw : ab)[LAYER || pass == 0 ? k / 2 : 0].get();
        *to = k & 1 ? t.y : t.x;
      } else {
#pragma unroll
        for (int h = 0; h < VEC / 4; ++h) {
          const int i = LAYER || pass == 0 ? k * VEC / 2 + 2 * h : 0;
          const float2 t = (pass == 0 ? aw : ab)[i].get(), u = (pass == 0 ? aw : ab)[LAYER || pass == 0 ? i + 1 : 0].get();
          reinterpret_cast<float4*>(to)[h] = make_float4(t.x, t.y, u.x, u.y);
        }
      }
    }
  }
  if (!side_by_side) return;
  __syncthreads();
  const int tid = threadIdx.y * tpr + l, threads = tpr * groups;
  for (int c = tid; c < a.D; c += threads) {
    float t = 0.0f, u = 0.0f;
    if (a.dw) {
      for (int g = 0; g < groups; ++g) t += shared[g * a.D + c];
    }
    if (LAYER && a.db) {
      for (int g = 0; g < groups; ++g) u += shared[(groups + g) * a.D + c];
    }
    if (a.cluster) {  // only this thread reads or writes column c of this block
      shared[c] = t;
      if (LAYER) shared[groups * a.D + c] = u;
    } else {
      if (a.dw) a.part_w[row + c] = t;
      if (LAYER && a.db) a.part_b[row + c] = u;
    }
  }
  if (!a.cluster) return;
  // The grid is one cluster: the blocks share out the columns and add one
  // another's sums in the order of their ranks.
  cluster_sync();
  const uint32_t at = smem_u32(shared), ranks = gridDim.x;
  for (int c = static_cast<int>(blockIdx.x) * threads + tid; c < a.D; c += static_cast<int>(ranks) * threads) {
    float t = 0.0f, u = 0.0f;
    for (uint32_t r = 0; r < ranks; ++r) {
      const uint32_t other = mapa_shared(at, r);
      t += load_cluster(other + 4u * c);
      if (LAYER) u += load_cluster(other + 4u * (groups * a.D + c));
    }
    if (a.dw) store_param(a.dw, a.p_type, c, t);
    if (LAYER && a.db) store_param(a.db, a.p_type, c, u);
  }
  cluster_sync();  // no block leaves while another reads its sums
}

// Rows too long for the registers of one block: grad_x by one block per row in
// two passes over it, the parameter gradients column-wise by cols_kernel.
template <typename TX, typename TY, int VEC, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) bwd_long_kernel(NormBwd a) {
  __shared__ float2 sm[MAX_THREADS / 32];
  const int64_t n = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n));
  const TY* dy = static_cast<const TY*>(a.dy) + a.gm.at(static_cast<int>(n));
  TX* dx = static_cast<TX*>(a.dx) + n * a.D;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const float rstd = a.rstd[n], mean = LAYER ? a.mean[n] : 0.0f;
  const int64_t first = static_cast<int64_t>(threadIdx.x) * VEC, step = static_cast<int64_t>(blockDim.x) * VEC;
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll 2
  for (int64_t c = first; c < a.D; c += step) {
    Vec<TX, VEC> xv;
    Vec<TY, VEC> gv;
    float w[VEC];
    xv.load(x + c);
    gv.load(dy + c);
    load_gain<LAYER, VEC>(a.w, a.p_type, a.offset, c, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float z = (xv.get(e) - mean) * rstd, g = gv.get(e) * w[e];
      if (LAYER) s.x += g;
      s.y += g * z;
    }
  }
  s = group_sum2<LAYER>(s, sm);
  s.x *= inv_d;
  s.y *= inv_d;
#pragma unroll 2
  for (int64_t c = first; c < a.D; c += step) {
    Vec<TX, VEC> xv;
    Vec<TY, VEC> gv;
    float w[VEC], o[VEC];
    xv.load(x + c);
    gv.load(dy + c);
    load_gain<LAYER, VEC>(a.w, a.p_type, a.offset, c, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float z = (xv.get(e) - mean) * rstd;
      o[e] = rstd * (gv.get(e) * w[e] - (s.x + z * s.y));
    }
    Vec<TX, VEC> out;
    out.set(o);
    out.store(dx + c);
  }
}

// Partial parameter gradients column-wise: a thread sums VEC columns over the
// rows blockIdx.y, blockIdx.y + gridDim.y, ...
template <typename TX, typename TY, int VEC, bool LAYER>
__global__ void __launch_bounds__(128) cols_kernel(NormBwd a) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * VEC;
  if (c >= a.D) return;
  float aw[VEC], ab[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    aw[e] = 0.0f;
    ab[e] = 0.0f;
  }
#pragma unroll 4
  for (int64_t n = blockIdx.y; n < a.N; n += gridDim.y) {
    Vec<TX, VEC> xv;
    Vec<TY, VEC> gv;
    xv.load(static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n)) + c);
    gv.load(static_cast<const TY*>(a.dy) + a.gm.at(static_cast<int>(n)) + c);
    const float rstd = a.rstd[n], mean = LAYER ? a.mean[n] : 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      aw[e] += gv.get(e) * ((xv.get(e) - mean) * rstd);
      if (LAYER) ab[e] += gv.get(e);
    }
  }
  const int64_t at = static_cast<int64_t>(blockIdx.y) * a.D + c;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if (a.dw) a.part_w[at + e] = aw[e];
    if (LAYER && a.db) a.part_b[at + e] = ab[e];
  }
}

// The parameter gradients from `parts` partial rows (0 parts: zeros).  A block
// adds 32 columns: its warps take the parts w, w + 32, ... in order (five of 152,
// all in flight at once), and warp 0 adds the warps in order.  blockIdx.y = 0:
// the weight's, 1: the bias's.
constexpr int REDUCE_WARPS = 32;
static __global__ void __launch_bounds__(32 * REDUCE_WARPS) reduce_kernel(const float* part_w, const float* part_b,
                                                                          int parts, int D, int p_type, void* dw,
                                                                          void* db) {
  __shared__ float ws[REDUCE_WARPS][32];
  wait_for_previous();
  void* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < D) {
#pragma unroll 5
    for (int p = threadIdx.y; p < parts; p += REDUCE_WARPS) s += part[static_cast<int64_t>(p) * D + c];
  }
  ws[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    s = 0.0f;
    for (int i = 0; i < REDUCE_WARPS; ++i) s += ws[i][threadIdx.x];
    store_param(out, p_type, c, s);
  }
}

// ------------------------------------------------------------------- launch
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads of a group that covers `vecs` vectors, K each.
inline int group_threads(int64_t vecs, int K) {
  const int64_t t = cdiv(vecs, K);
  if (t > 32) return static_cast<int>(cdiv(t, 32) * 32);
  int p = 1;
  while (p < t) p *= 2;
  return p;
}

template <typename TX, typename TY, int VEC, int K, bool LAYER>
cudaError_t run_fwd_few(const NormFwd& a, int64_t vecs, cudaStream_t s) {
  fwd_few_kernel<TX, TY, VEC, K, LAYER><<<static_cast<unsigned>(a.N), group_threads(vecs, K), 0, s>>>(a);
  return cudaGetLastError();
}

constexpr int MAX_SMEM = 227 * 1024 - 2048;   // dynamic shared memory of a block, beside what the kernels declare
constexpr int PLAIN_SMEM = 48 * 1024 - 2048;  // of a block that has not asked for more

template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER>
cudaError_t run_fwd(const NormFwd& a, int tpr, cudaStream_t s) {
  const int smem = static_cast<int>(sizeof(float)) * a.D * (LAYER ? 2 : 1);
  // Two blocks of 256 threads fill an SM's registers; where their parameters do not fit twice, one of 512.
  const bool pair = 2 * (smem + 2048) <= MAX_SMEM;
  const int groups = std::max(1, (pair ? 256 : MAX_THREADS) / tpr);
  const int per_sm = std::max(1, MAX_THREADS / (tpr * groups));
  const int grid = static_cast<int>(std::min<int64_t>(cdiv(a.N, groups), a.sms * per_sm));
  if (smem > PLAIN_SMEM) {
    const cudaError_t e = cudaFuncSetAttribute(fwd_kernel<TX, TY, VEC, K, KF, LAYER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  fwd_kernel<TX, TY, VEC, K, KF, LAYER><<<grid, dim3(tpr, groups), smem, s>>>(a);
  return cudaGetLastError();
}

template <typename TX, typename TY, int VEC, bool LAYER>
cudaError_t fwd(const NormFwd& a, cudaStream_t s, int* launches) {
  if (a.N == 0) return cudaSuccess;
  ++*launches;
  const int64_t vecs = a.D / VEC;
  if (a.N <= a.sms) {
    if (vecs <= MAX_THREADS) return run_fwd_few<TX, TY, VEC, 1, LAYER>(a, vecs, s);
    if (vecs <= 4 * MAX_THREADS) return run_fwd_few<TX, TY, VEC, 4, LAYER>(a, vecs, s);
  }
  const bool fits = static_cast<int64_t>(sizeof(float)) * a.D * (LAYER ? 2 : 1) <= MAX_SMEM;
  if constexpr (VEC > 1) {
    const int tpr = group_threads(vecs, vecs <= 64 ? 4 : 8);
    if (fits && tpr <= MAX_THREADS) {
      switch (cdiv(vecs, tpr)) {  // vectors a thread; all but its last are there in every thread
        case 1: return run_fwd<TX, TY, VEC, 1, 0, LAYER>(a, tpr, s);
        case 2: return run_fwd<TX, TY, VEC, 2, 1, LAYER>(a, tpr, s);
        case 3: return run_fwd<TX, TY, VEC, 3, 2, LAYER>(a, tpr, s);
        case 4: return run_fwd<TX, TY, VEC, 4, 3, LAYER>(a, tpr, s);
        case 5: return run_fwd<TX, TY, VEC, 5, 4, LAYER>(a, tpr, s);
        case 6: return run_fwd<TX, TY, VEC, 6, 5, LAYER>(a, tpr, s);
        case 7: return run_fwd<TX, TY, VEC, 7, 6, LAYER>(a, tpr, s);
        default: return run_fwd<TX, TY, VEC, 8, 7, LAYER>(a, tpr, s);
      }
    }
  } else {
    const int K = vecs <= 32 ? 4 : vecs <= 128 ? 8 : vecs <= 512 ? 16 : 32;
    const int tpr = group_threads(vecs, K);
    if (fits && tpr <= MAX_THREADS) {
      switch (K) {
        case 4: return run_fwd<TX, TY, VEC, 4, 0, LAYER>(a, tpr, s);
        case 8: return run_fwd<TX, TY, VEC, 8, 4, LAYER>(a, tpr, s);
        case 16: return run_fwd<TX, TY, VEC, 16, 8, LAYER>(a, tpr, s);
        default: return run_fwd<TX, TY, VEC, 32, 16, LAYER>(a, tpr, s);
      }
    }
  }
  fwd_long_kernel<TX, TY, VEC, LAYER><<<static_cast<unsigned>(a.N), MAX_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

constexpr int CLUSTER = 8;  // blocks, the portable limit
#ifndef CLUSTER_ROWS
#define CLUSTER_ROWS 1
#endif

template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER>
cudaError_t run_bwd(const NormBwd& a, int tpr, int* parts, cudaStream_t s) {
  // Where the sums of 24 values and the two rows fit beside each other: not those of a layer norm.
  constexpr bool PREFETCH = K * VEC <= (LAYER ? 16 : 24);
  const int groups = std::max(1, bwd_threads<TX, VEC, K, LAYER>() / tpr);
  NormBwd b = a;
  b.cluster = (a.dw || a.db) && a.N <= static_cast<int64_t>(CLUSTER_ROWS) * CLUSTER * groups;
  int blocks = static_cast<int>(std::min<int64_t>({NORM_MAX_PARTS, a.sms, cdiv(a.N, groups)}));
  if (b.cluster) {
    int size = 1;
    while (size < blocks && size < CLUSTER) size *= 2;
    blocks = size;
  }
  *parts = b.cluster ? 0 : blocks;
  auto kernel = bwd_kernel<TX, TY, VEC, K, KF, LAYER, PREFETCH>;
  const int smem = static_cast<int>(sizeof(float)) * a.D * ((groups > 1 || b.cluster) && LAYER ? 2 * groups : groups);
  if (smem > PLAIN_SMEM) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = b.cluster ? static_cast<unsigned>(blocks) : 1u;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(tpr, groups);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, b);
}

// Launches bwd_kernel for rows that the registers of one block hold; false for longer ones.
template <typename TX, typename TY, int VEC, bool LAYER>
bool bwd_in_registers(const NormBwd& a, int* parts, cudaStream_t s, cudaError_t* e) {
  const int64_t vecs = a.D / VEC;
  if constexpr (VEC > 1) {
    constexpr int K = 16 / VEC;
    const int most = bwd_threads<TX, VEC, K, LAYER>();
    int tpr = group_threads(vecs, K);
    if (tpr <= most) {
      switch (cdiv(vecs, tpr)) {  // vectors a thread; all but its last are there in every thread
        case 1: *e = run_bwd<TX, TY, VEC, 1, 0, LAYER>(a, tpr, parts, s); break;
        case 2: *e = run_bwd<TX, TY, VEC, 2, 1, LAYER>(a, tpr, parts, s); break;
        case 3: *e = run_bwd<TX, TY, VEC, K < 3 ? 2 : 3, K < 3 ? 1 : 2, LAYER>(a, tpr, parts, s); break;
        default: *e = run_bwd<TX, TY, VEC, K, K - 1, LAYER>(a, tpr, parts, s); break;
      }
      return true;
    }
    if (vecs > 2 * K * MAX_THREADS) return false;
    // as few values a thread as 512 threads allow
    const bool most_values = vecs > 3 * K / 2 * MAX_THREADS;
    tpr = group_threads(vecs, most_values ? 2 * K : 3 * K / 2);
    *e = most_values ? run_bwd<TX, TY, VEC, 2 * K, 3 * K / 2, LAYER>(a, tpr, parts, s)
                     : run_bwd<TX, TY, VEC, 3 * K / 2, K, LAYER>(a, tpr, parts, s);
  } else {
    const int K = vecs <= 32 ? 4 : vecs <= 16 * MAX_THREADS ? 16 : 32;
    const int tpr = group_threads(vecs, K);
    if (tpr > MAX_THREADS) return false;
    switch (K) {
      case 4: *e = run_bwd<TX, TY, VEC, 4, 0, LAYER>(a, tpr, parts, s); break;
      case 16: *e = run_bwd<TX, TY, VEC, 16, 8, LAYER>(a, tpr, parts, s); break;
      default: *e = run_bwd<TX, TY, VEC, 32, 16, LAYER>(a, tpr, parts, s); break;
    }
  }
  return true;
}

template <typename TX, typename TY, int VEC, bool LAYER>
cudaError_t bwd(const NormBwd& a, cudaStream_t s, int* launches) {
  int parts = 0;
  if (a.N > 0 && (a.dx || a.dw || a.db)) {
    ++*launches;
    cudaError_t e = cudaSuccess;
    if (!bwd_in_registers<TX, TY, VEC, LAYER>(a, &parts, s, &e)) {
      if (a.dx) bwd_long_kernel<TX, TY, VEC, LAYER><<<static_cast<unsigned>(a.N), MAX_THREADS, 0, s>>>(a);
      if (a.dw || a.db) {
        const int64_t tiles = cdiv(a.D / VEC, 128);
        parts = static_cast<int>(
            std::min<int64_t>({NORM_MAX_PARTS, cdiv(a.N, 8), std::max<int64_t>(1, 8 * a.sms / tiles)}));
        *launches += a.dx ? 1 : 0;
        cols_kernel<TX, TY, VEC, LAYER>
            <<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(parts)), 128, 0, s>>>(a);
      }
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  if ((!a.dw && !a.db) || (a.N > 0 && parts == 0)) return cudaSuccess;  // parts == 0: the cluster has written them
  ++*launches;
  return launch_after(reduce_kernel, dim3(static_cast<unsigned>(cdiv(a.D, 32)), LAYER ? 2 : 1), dim3(32, REDUCE_WARPS),
                      s, a.part_w, a.part_b, parts, a.D, a.p_type, a.dw, a.db);
}

template <typename TX, typename TY>
cudaError_t fwd_any(const NormFwd& a, bool layer, bool wide, cudaStream_t s, int* launches) {
  constexpr int VEC = 16 / sizeof(TX);
  if (layer) return wide ? fwd<TX, TY, VEC, true>(a, s, launches) : fwd<TX, TY, 1, true>(a, s, launches);
  return wide ? fwd<TX, TY, VEC, false>(a, s, launches) : fwd<TX, TY, 1, false>(a, s, launches);
}

template <typename TX, typename TY>
cudaError_t bwd_any(const NormBwd& a, bool layer, bool wide, cudaStream_t s, int* launches) {
  constexpr int VEC = 16 / sizeof(TX);
  if (layer) return wide ? bwd<TX, TY, VEC, true>(a, s, launches) : bwd<TX, TY, 1, true>(a, s, launches);
  return wide ? bwd<TX, TY, VEC, false>(a, s, launches) : bwd<TX, TY, 1, false>(a, s, launches);
}

}  // namespace norm
}  // namespace cce

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
// Rows whose starts are not 16-byte aligned (odd widths, views) are read and
// written in aligned vectors all the same (SHIFTED): vector v of row n covers the
// columns v * VEC - s ... for a row whose start lies s elements behind a vector's,
// and only the row's two end vectors are partial.  s is the output's; where a
// row of an input has another s (REALIGNED), each of the output's vectors is
// joined from the two of the input's that hold its columns.
//
// A row belongs to a group of threadIdx.x = 0 .. tpr - 1 (tpr a power of two up
// to 32, or a multiple of 32); a block has blockDim.y groups.  Thread l of a
// group holds the vectors l, l + tpr, ..., K of them.
#pragma once

#include <algorithm>
#include <type_traits>

#include "elements.cuh"
#include "norm.h"
#include "ptx.cuh"

namespace cce {
namespace norm {

constexpr int MAX_THREADS = 512;

// Over `width` neighbouring lanes (a power of two); every step is there, those that cross groups add nothing.
__device__ __forceinline__ float lanes_sum(float v, int width) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, v, o);
    if (o < width) v += t;
  }
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

// Slots in shared memory for one value of every warp of a block, each group's
// padded to a multiple of four.
constexpr int slots(int threads) { return threads / 16; }
__device__ __forceinline__ int group_slots() { return ((blockDim.x >> 5) + 3) & ~3; }

// Lane 0 of a warp puts its value, of the last warp zeros behind it too.
__device__ __forceinline__ void put_slot(float* sm, float v) {
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  sm[warp] = v;
  if (warp == warps - 1) {
    for (int i = warps; i & 3; ++i) sm[i] = 0.0f;
  }
}

// Sum over the group; sm: the group's slots.
__device__ __forceinline__ float group_sum(float v, float* sm) {
  const int tpr = blockDim.x;
  v = lanes_sum(v, min(tpr, 32));
  if (tpr <= 32) return v;
  if ((threadIdx.x & 31) == 0) put_slot(sm, v);
  group_sync();
  float t = 0.0f;
#pragma unroll 1
  for (int i = 0; i < tpr >> 5; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(sm + i);
    t += (q.x + q.y) + (q.z + q.w);
  }
  return t;
}

// Of two values; sm: the group's slots for the first, `second` floats on those for the second.
__device__ __forceinline__ float2 group_sum2(float2 v, float* sm, int second) {
  const int tpr = blockDim.x;
  v.x = lanes_sum(v.x, min(tpr, 32));
  v.y = lanes_sum(v.y, min(tpr, 32));
  if (tpr <= 32) return v;
  if ((threadIdx.x & 31) == 0) {
    put_slot(sm, v.x);
    put_slot(sm + second, v.y);
  }
  group_sync();
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll 1
  for (int i = 0; i < tpr >> 5; i += 4) {
    const float4 p = *reinterpret_cast<const float4*>(sm + i), q = *reinterpret_cast<const float4*>(sm + second + i);
    t.x += (p.x + p.y) + (p.z + p.w);
    t.y += (q.x + q.y) + (q.z + q.w);
  }
  return t;
}

// The gain and the bias of VEC columns; SOME: of the first n, the others 0.  CONSTANT: by load_constant().
template <bool LAYER, int VEC, bool SOME = false, bool CONSTANT = false>
__device__ __forceinline__ void load_gain(const void* w, int p_type, float offset, int64_t c, float (&g)[VEC],
                                          int n = VEC) {
  if (w) {
    load_param<VEC, SOME, CONSTANT>(w, p_type, c, g, n);
    if (!LAYER) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (!SOME || e < n) g[e] += offset;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = 1.0f;
  }
}

template <bool LAYER, int VEC, bool SOME = false, bool CONSTANT = false>
__device__ __forceinline__ void load_bias(const void* b, int p_type, int64_t c, float (&f)[VEC], int n = VEC) {
  if (LAYER && b) {
    load_param<VEC, SOME, CONSTANT>(b, p_type, c, f, n);
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

// Where a row lies in a thread's vectors.  Every row has the first KF vectors of
// every thread, so that only the others are checked.
template <int VEC, int KF, Access A>
struct Place {
  static constexpr bool REALIGNED = A == Access::REALIGNED, SHIFTED = REALIGNED || A == Access::SHIFTED;
  int D, vecs;    // columns; vectors that a row may touch
  int first;      // s of row 0
  int s = 0;      // columns by which the row starts inside vector 0
  int used;       // vectors that this row touches

  __device__ __forceinline__ Place(int d, int shift)
      : D(d), vecs(SHIFTED ? (d + 2 * VEC - 2) / VEC : d / VEC), first(REALIGNED ? shift : 0), used(vecs) {}
  __device__ __forceinline__ void row(int64_t n) {
    if constexpr (SHIFTED) {
      s = static_cast<int>(n * (D & (VEC - 1)) + first) & (VEC - 1);
      used = (D + s + VEC - 1) / VEC;
    }
  }
  __device__ __forceinline__ int vec(int k) const { return static_cast<int>(threadIdx.x + k * blockDim.x); }
  __device__ __forceinline__ bool has(int k) const { return k < KF || vec(k) < used; }
  __device__ __forceinline__ int column(int k) const { return vec(k) * VEC - s; }  // of the vector's first element
  // The elements lo .. hi - 1 of vector k are the row's.
  __device__ __forceinline__ int lo(int k) const { return SHIFTED ? max(0, -column(k)) : 0; }
  __device__ __forceinline__ int hi(int k) const { return SHIFTED ? min(VEC, D - column(k)) : VEC; }
  __device__ __forceinline__ bool whole(int k) const {
    return !SHIFTED || (column(k) >= 0 && column(k) + VEC <= D);
  }

  // The s of an input's row n.
  template <typename T>
  __device__ __forceinline__ int own(const T* row) const {
    return REALIGNED ? static_cast<int>(reinterpret_cast<uintptr_t>(row) / sizeof(T)) & (VEC - 1) : s;
  }
  __device__ __forceinline__ bool has(int k, int o) const {  // with s = o
    return REALIGNED ? k < KF || vec(k) * VEC - o < D : has(k);
  }
  // Whether the vector from column c of row n on, which starts at element `at` of
  // `end`, may be read whole: no memory need be around the matrix.
  __device__ __forceinline__ bool readable(int c, bool last, int64_t at, int64_t end) const {
    if (!SHIFTED || (!REALIGNED && !last) || (c >= 0 && c + VEC <= D)) return true;
    return REALIGNED && at + c >= 0 && at + c + VEC <= end;
  }
  // The row's vector from column c on.  It brings its neighbours' elements: trim()
  // drops them, once it is used (here it would wait for the load).
  template <typename T>
  __device__ __forceinline__ void load(Vec<T, VEC>& v, const T* row, int c, bool last, int64_t at, int64_t end) const {
    if (readable(c, last, at, end)) {
      v.load(row + c);
    } else {
      v.load_some(row + c, max(0, -c), min(VEC, D - c));
    }
  }
  template <typename T>
  __device__ __forceinline__ void trim(Vec<T, VEC>& v, int k) const {
    if (SHIFTED && !whole(k)) v.keep(lo(k), hi(k));
  }
  template <typename T>
  __device__ __forceinline__ void store(const Vec<T, VEC>& v, T* p, int k) const {
    if (whole(k)) {
      v.store(p + column(k));
    } else {
      v.store_some(p + column(k), lo(k), hi(k));
    }
  }

  // Parameters in shared memory as fp32.  A vector's float4 quarters (SHIFTED: its
  // elements) lie `vecs` apart, so that a warp's reads fall on consecutive addresses.
  __device__ __forceinline__ int param_floats() const { return SHIFTED ? VEC * vecs : D; }
  __device__ __forceinline__ void put_param(float* sm, int c, const float (&f)[VEC]) const {  // vector c of the D columns
    if constexpr (SHIFTED || VEC == 1) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) sm[e * vecs + c] = f[e];
    } else {
#pragma unroll
      for (int h = 0; h < VEC / 4; ++h)
        reinterpret_cast<float4*>(sm)[h * vecs + c] = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
    }
  }
  // Of the columns of vector k; any value for those that are not the row's.
  __device__ __forceinline__ void get_param(const float* sm, int k, float (&f)[VEC]) const {
    const int v = vec(k);
    if constexpr (SHIFTED || VEC == 1) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int at = e - s;  // column v * VEC + at; never before the first, never past the last of all planes
        f[e] = sm[(at & (VEC - 1)) * vecs + v + (at < 0 ? -1 : 0)];
      }
    } else {
#pragma unroll
      for (int h = 0; h < VEC / 4; ++h) {
        const float4 q = reinterpret_cast<const float4*>(sm)[h * vecs + v];
        f[4 * h] = q.x;
        f[4 * h + 1] = q.y;
        f[4 * h + 2] = q.z;
        f[4 * h + 3] = q.w;
      }
    }
  }
  // All of a block's threads: the parameters of the D columns; what `load` makes of none past them.
  template <typename Load>
  __device__ __forceinline__ void fill(float* sm, Load load) const {
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
    for (int c = tid; c < vecs; c += threads) {
      float f[VEC];
      load(static_cast<int64_t>(c) * VEC, f, min(VEC, D - c * VEC));
      put_param(sm, c, f);
    }
  }
};

// ------------------------------------------------------------------ forward
// Few rows: a block of up to 512 threads per row, so that a row's loads are all
// in flight at once; parameters are loaded beside them.  Bound by latency, a
// load and two block sums: 2.1 us for one row of 896 bf16 values, launch included.
template <typename TX, typename TY, int VEC, int K, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) fwd_few_kernel(NormFwd a) {
  __shared__ __align__(16) float sm[2][slots(MAX_THREADS)];
  const int l = threadIdx.x, tpr = blockDim.x;
  const int64_t n = blockIdx.x;
  const TX* x = static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n));
  let_next_start();
  wait_for_previous();
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
//
// Bound by memory.  bf16 65,536 x 2,048: RMS norm 86 us (6.2 TB/s), layer norm,
// with a second sum and a bias, 94 us (5.7 TB/s), a copy of the same bytes 82 us;
// 8,192 x 2,304: 15.0 and 16.8 us, a copy 13.  With a bounds check on every vector
// instead of the last one 99 us; with one block of 128 threads a row and no row
// ahead 254 us.  Rows spread over more threads pay more for their sums: 16,384 x
// 4,096 takes 46 us with 64 values a thread, 48 us with 32, 64 us with 16.
//
// The bound of one block an SM stands for the 512 threads an SM that run_fwd launches: without it the compiler held
// some variants to 64 registers, and they spilled (fp32 32,768 x 561 into bf16 33.6 us, with it 29.4).
template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER, Access A>
__global__ void __launch_bounds__(MAX_THREADS, 1) fwd_kernel(NormFwd a) {
  constexpr bool REALIGNED = A == Access::REALIGNED, SHIFTED = REALIGNED || A == Access::SHIFTED;
  constexpr int E = K * VEC / 2;
  extern __shared__ __align__(16) float gain[];  // then the bias of a layer norm
  __shared__ __align__(16) float sm[4][slots(MAX_THREADS)];
  const int groups = blockDim.y, slot = threadIdx.y * group_slots();
  const int step = gridDim.x * groups;
  Place<VEC, KF, A> next(a.D, a.shift);
  float* bias = gain + next.param_floats();
  Vec<TX, VEC> xv[K];
#pragma unroll
  for (int k = 0; k < K; ++k) xv[k].zero();
  auto load_row = [&](int64_t n) {
    if (n >= a.N) return;
    next.row(n);
    const int64_t at = a.xm.at(static_cast<int>(n));
    const TX* x = static_cast<const TX*>(a.x) + at;
    const int o = next.own(x);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (next.has(k, o)) {
        next.load(xv[k], x, next.vec(k) * VEC - o, n == a.N - 1, at, a.x_end);
      } else if (SHIFTED) {
        xv[k].zero();
      }
    }
  };
  // The vectors of a row of x as y's: the neighbours of a thread's vectors are in L1 (16,368 x 2,049 58 us for a
  // layer norm; 41 where no row needs it).
  auto realign = [&](int64_t n, const Place<VEC, KF, A>& place) {
    const int64_t at = a.xm.at(static_cast<int>(n));
    const TX* x = static_cast<const TX*>(a.x) + at;
    const int o = place.own(x), by = o - place.s;
    if (by == 0) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (place.vec(k) + (by < 0 ? -1 : 1)) * VEC - o;
      Vec<TX, VEC> other;
      other.zero();
      if (c > -VEC && c < a.D) place.load(other, x, c, false, at, a.x_end);
      if (by < 0) {
        xv[k].join(other, xv[k], by + VEC);
      } else {
        xv[k].join(xv[k], other, by);
      }
    }
  };
  let_next_start();
  wait_for_previous();
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
  load_row(base + threadIdx.y);
  next.fill(gain, [&](int64_t c, auto& f, int n) {
    load_gain<LAYER, VEC, SHIFTED>(a.w, a.p_type, a.offset, c, f, n);
  });
  if (LAYER) {
    next.fill(bias, [&](int64_t c, auto& f, int n) { load_bias<LAYER, VEC, SHIFTED>(a.b, a.p_type, c, f, n); });
  }
  __syncthreads();
  const float fd = static_cast<float>(a.D);
  int buf = 0;
  for (; base < a.N; base += step) {
    const int64_t n = base + threadIdx.y;
    const Place<VEC, KF, A> place = next;
    if constexpr (REALIGNED) {
      if (n < a.N) realign(n, place);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) place.trim(xv[k], k);
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
      if constexpr (VEC == 1) {  // columns that are not there would add mean^2
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float2 f = d[i].get();
          d[i] = Pair::of(place.has(2 * i) ? f.x : 0.0f, place.has(2 * i + 1) ? f.y : 0.0f);
        }
      } else if constexpr (SHIFTED) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!place.whole(k)) {
            const int lo = place.lo(k), hi = place.hi(k);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
              const float2 f = d[k * VEC / 2 + i].get();
              d[k * VEC / 2 + i] = Pair::of(2 * i >= lo && 2 * i < hi ? f.x : 0.0f,
                                            2 * i + 1 >= lo && 2 * i + 1 < hi ? f.y : 0.0f);
            }
          }
        }
      }
    }
    Pair q[2] = {Pair::both(0.0f), Pair::both(0.0f)};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      // elsewhere a vector that is not there is 0
      if (!LAYER || VEC == 1 || SHIFTED || place.has(2 * i / VEC)) q[i & 1] = fma(d[i], d[i], q[i & 1]);
    }
    const float rstd = 1.0f / sqrtf(group_sum(add(q[0], q[1]).sum(), sm[buf + 1] + slot) / fd + a.eps);
    buf ^= 2;  // the other slots for the next row: a slower warp may still read these
    if (n >= a.N) continue;
    if (threadIdx.x == 0) {
      if (LAYER && a.mean) a.mean[n] = mean;
      if (a.rstd) a.rstd[n] = rstd;
    }
    TY* y = static_cast<TY*>(a.y) + n * a.D;
    const Pair r = Pair::both(rstd);
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = mul(d[i], r);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (place.has(k)) {
        float w[VEC], b[VEC], o[VEC];
        place.get_param(gain, k, w);
        if (LAYER) place.get_param(bias, k, b);
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
        place.store(out, y, k);
      }
    }
  }
}

// Rows too long for the registers of one block: one block per row, which
// reads it once per sum and once more to write (from L2 after the first time).
// These are rows of more than 16,384 fp32 columns, of more than 32,768 16-bit ones
// for an RMS norm, and of more than 28,800 for a layer norm, whose gain and bias
// fill shared memory first.
// bf16 2,048 x 30,000, layer norm: 71 us (3.5 TB/s of the bytes read and written
// once); 2,048 x 33,000, RMS norm: 52 us; 2,048 x 33,001, by elements, 187 us.
template <typename TX, typename TY, int VEC, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) fwd_long_kernel(NormFwd a) {
  __shared__ __align__(16) float sm[2][slots(MAX_THREADS)];
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
      v.load_constant(x + c);
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
    v.load_constant(x + c);
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
    v.load_constant(x + c);
    float w[VEC], b[VEC], o[VEC];
    load_gain<LAYER, VEC, false, true>(a.w, a.p_type, a.offset, c, w);
    load_bias<LAYER, VEC, false, true>(a.b, a.p_type, c, b);
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
// the forward.  The next rows wait in a ring of shared memory: each thread copies
// its own vectors there, so a thread waits for nothing but its own copies.
//
// Bound by memory, a layer norm by the registers that keep fewer rows in flight:
// bf16 65,536 x 2,048, 805 MB, RMS norm 119 us (6.8 TB/s), layer norm 137 us (5.9
// TB/s); 8,192 x 2,304 24 and 27 us, 3 us of it the parameters' gradients.  A
// layer norm of 12,289 to 16,384 columns, 32 values a thread with both sums,
// spills 68 to 348 bytes a thread: 4,096 x 16,384 110 us in bf16 (59 at a copy's
// rate) and 180 in fp32 (119), 4,096 x 12,288 59 and 105.
// With the next row in registers instead of the ring 125 and 142 us; with three
// or four rows in it 120 and 138.  Odd widths pay for their partial vectors: 16,384
// x 1,001 29 and 34 us, x 1,024 22 and 25 us.
//
// Threads of a block: as many as the sums leave registers for.  A layer norm's
// have the bias's beside the weight's; its rows of 257 to 320 threads fit twice
// in 640 (bf16 8,192 x 5,120: 56 us against 65), where fewer registers cost the
// others 0.5 us a call.
template <typename TX, int VEC, int K, bool LAYER>
constexpr int bwd_threads() {
  return !LAYER && sizeof(TX) == 2 && VEC > 1 && K * VEC <= 16 ? 768 : 512;
}
constexpr int WIDER = 640;
// A group of several warps has the barrier of its number plus one, of 16 that there are.
static_assert(768 / 64 + 1 <= 16, "barriers of a block");
// Rows in the ring: one where a thread holds more than 16 values, none for single elements.
template <int VEC, int K>
constexpr int bwd_ring() {
  return VEC == 1 ? 0 : K * VEC > 16 ? 1 : 2;
}
template <typename TX, typename TY, int VEC, int K, int THREADS>
constexpr int bwd_ring_bytes() {
  return bwd_ring<VEC, K>() * THREADS * K * VEC * static_cast<int>(sizeof(TX) + sizeof(TY));
}

__device__ __forceinline__ float load_cluster(uint32_t addr) {
  float f;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(addr) : "memory");
  return f;
}

template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER, Access A, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) bwd_kernel(NormBwd a) {
  constexpr bool REALIGNED = A == Access::REALIGNED, SHIFTED = REALIGNED || A == Access::SHIFTED;
  constexpr int E = K * VEC / 2, RING = bwd_ring<VEC, K>();
  constexpr int AHEAD = RING > 0 ? RING : 1;  // rows whose statistics are loaded
  extern __shared__ __align__(16) float dynamic[];  // the ring, then the gain; at the end the groups' sums
  Vec<TX, VEC>* const ring_x = reinterpret_cast<Vec<TX, VEC>*>(dynamic);  // [RING][K][THREADS]
  Vec<TY, VEC>* const ring_g = reinterpret_cast<Vec<TY, VEC>*>(ring_x + RING * K * THREADS);
  float* const gain = dynamic + bwd_ring_bytes<TX, TY, VEC, K, THREADS>() / sizeof(float);
  constexpr int SLOTS = slots(THREADS);
  __shared__ __align__(16) float sm[2][2][SLOTS];
  const int l = threadIdx.x, tpr = blockDim.x, groups = blockDim.y, slot = threadIdx.y * group_slots();
  const int own = threadIdx.y * tpr + l;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  const float inv_d = 1.0f / static_cast<float>(a.D);

  // A group's rows are all shifted alike: there is one row, or `step` is a multiple of VEC.
  Place<VEC, KF, A> place(a.D, a.shift);
  float mean[AHEAD], rstd[AHEAD];
  auto load_stats = [&](int64_t n, int i) {
    mean[i] = LAYER && n < a.N ? a.mean[n] : 0.0f;
    rstd[i] = n < a.N ? a.rstd[n] : 0.0f;
  };
  // Requests row n into place `at` of the ring.
  auto request_from = [&](auto* ring, const auto* m, bool last, int64_t row, int64_t end, int at) {
    using V = std::remove_reference_t<decltype(*ring)>;
    m += row;
    const int o = place.own(m);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!place.has(k, o)) continue;
      V* const to = ring + (at * K + k) * THREADS + own;
      const int c = place.vec(k) * VEC - o;
      if (place.readable(c, last, row, end)) {
        copy_async<sizeof(V)>(to, m + c);
      } else {
        to->load_some(m + c, max(0, -c), min(VEC, a.D - c));
      }
    }
  };
  auto request = [&](int64_t n, int at) {
    if (n < a.N) {
      const bool last = n == a.N - 1;
      request_from(ring_x, static_cast<const TX*>(a.x), last, a.xm.at(static_cast<int>(n)), a.x_end, at);
      request_from(ring_g, static_cast<const TY*>(a.dy), last, a.gm.at(static_cast<int>(n)), a.dy_end, at);
    }
    end_copy_group();
  };
  // Vector k of an input whose rows are shifted by `by` more than dx's.
  auto take = [&](auto& v, const auto* ring, int at, int k, int by) {
    const auto* const mine = ring + (at * K + k) * THREADS + own;
    if (!REALIGNED || by == 0) {
      v = *mine;
      return;
    }
    // The neighbouring vector; what lies before the first and behind the last is trimmed.
    int to = by < 0 ? -1 : 1, k2 = k;
    if (l + to < 0 || l + to >= tpr) {
      k2 += to;
      to -= to * tpr;
    }
    const auto* const other = k2 < 0 || k2 >= K ? mine : ring + (at * K + k2) * THREADS + own + to;
    if (by < 0) {
      v.join(*other, *mine, by + VEC);
    } else {
      v.join(*mine, *other, by);
    }
  };
  // The threads that share a row's vectors.
  auto row_sync = [&] {
    if (tpr > 32) {
      group_sync();
    } else {
      __syncwarp();
    }
  };
  let_next_start();
  wait_for_previous();
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
  place.row(base + threadIdx.y);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    if constexpr (RING > 0) request(base + threadIdx.y + i * step, i);
    load_stats(base + threadIdx.y + i * step, i);
  }
  place.fill(gain, [&](int64_t c, auto& f, int n) {
    load_gain<LAYER, VEC, SHIFTED>(a.w, a.p_type, a.offset, c, f, n);
  });
  __syncthreads();

  Pair aw[E], ab[LAYER ? E : 1];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    aw[i] = Pair::both(0.0f);
    if (LAYER) ab[i] = Pair::both(0.0f);
  }
  int buf = 0, at = 0;
  for (; base < a.N; base += step) {
    const int64_t n = base + threadIdx.y;
    Vec<TX, VEC> x[K];
    Vec<TY, VEC> g[K];
    const float row_mean = mean[0], row_rstd = rstd[0];
    if constexpr (RING > 0) wait_copy_groups<RING - 1>();
    int by_x = 0, by_g = 0;
    if constexpr (REALIGNED) {
      row_sync();  // the other threads' copies are there too
      if (n < a.N) {
        by_x = place.own(static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n))) - place.s;
        by_g = place.own(static_cast<const TY*>(a.dy) + a.gm.at(static_cast<int>(n))) - place.s;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k].zero();
      g[k].zero();  // a row of zeros adds nothing
      if (n < a.N && place.has(k)) {
        if constexpr (RING > 0) {
          take(x[k], ring_x, at, k, by_x);
          take(g[k], ring_g, at, k, by_g);
          place.trim(x[k], k);
          place.trim(g[k], k);
        } else {
          x[k].load(static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n)) + place.column(k));
          g[k].load(static_cast<const TY*>(a.dy) + a.gm.at(static_cast<int>(n)) + place.column(k));
        }
      }
    }
    if constexpr (RING > 0) {
      if (REALIGNED) row_sync();  // and have been read
      request(n + RING * step, at);
      at = at + 1 == RING ? 0 : at + 1;
    }
#pragma unroll
    for (int i = 0; i + 1 < AHEAD; ++i) {
      mean[i] = mean[i + 1];
      rstd[i] = rstd[i + 1];
    }
    load_stats(n + AHEAD * step, AHEAD - 1);
    // z = (x - mean) rstd: the difference loses next to nothing where x is near the mean.  As x rstd - mean rstd, one
    // instruction less, every z of a row would carry the rounding of mean rstd.
    const Pair r = Pair::both(row_rstd), m = Pair::both(-row_mean);
    float2 s;
    {
      Pair s1 = Pair::both(0.0f), s2 = Pair::both(0.0f);
      auto gather = [&](int i, Pair w) {
        const Pair xp = pair_of<TX, VEC, K>(x, i), dp = pair_of<TY, VEC, K>(g, i);
        const Pair z = mul(LAYER ? add(xp, m) : xp, r);
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
          gather(k / 2, Pair::of(gain[place.has(k) ? place.vec(k) : 0],
                                 gain[place.has(k + 1) ? place.vec(k + 1) : 0]));
        }
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!place.has(k)) continue;
          float w[VEC];
          place.get_param(gain, k, w);
#pragma unroll
          for (int i = 0; i < VEC / 2; ++i) gather(k * VEC / 2 + i, Pair::of(w[2 * i], w[2 * i + 1]));
        }
      }
      s = make_float2(LAYER ? s1.sum() : 0.0f, s2.sum());
    }
    if (!a.dx) continue;
    s = LAYER ? group_sum2(s, sm[buf][0] + slot, SLOTS) : make_float2(0.0f, group_sum(s.y, sm[buf][0] + slot));
    buf ^= 1;  // the other slots for the next row: a slower warp may still read these
    if (n >= a.N) continue;
    TX* dx = static_cast<TX*>(a.dx) + n * a.D;
    const Pair c1 = Pair::both(-s.x * inv_d * row_rstd), c2 = Pair::both(-s.y * inv_d * row_rstd);
    // rstd (g - sum(g) / D - z sum(g z) / D)
    auto grad = [&](int i, Pair w) {
      const Pair xp = pair_of<TX, VEC, K>(x, i), dp = pair_of<TY, VEC, K>(g, i);
      const Pair z = mul(LAYER ? add(xp, m) : xp, r);
      return fma(mul(dp, w), r, LAYER ? fma(z, c2, c1) : mul(z, c2)).get();
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!place.has(k)) continue;
      float w[VEC], f[VEC];
      place.get_param(gain, k, w);
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
      place.store(out, dx, k);
    }
  }

  // Several groups: their sums side by side in shared memory (the weight's, then
  // the bias's), added in order.  One group: straight into the partial row.
  if (!a.dw && !a.db) return;
  const bool side_by_side = SHIFTED || groups > 1;
  float* const sums = dynamic;
  if (side_by_side) __syncthreads();  // the gain and the ring have been read
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.D;
#pragma unroll
  for (int pass = 0; pass < (LAYER ? 2 : 1); ++pass) {
    if (!(pass == 0 ? a.dw : a.db)) continue;
    float* part =
        side_by_side ? sums + (pass * groups + threadIdx.y) * a.D : (pass == 0 ? a.part_w : a.part_b) + row;
    auto value = [&](int i) { return (pass == 0 ? aw : ab)[LAYER || pass == 0 ? i : 0].get(); };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!place.has(k)) continue;
      float* to = part + place.column(k);
      if constexpr (VEC == 1) {
        const float2 t = value(k / 2);
        *to = k & 1 ? t.y : t.x;
      } else if constexpr (SHIFTED) {
        const int lo = place.lo(k), hi = place.hi(k);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 t = value(k * VEC / 2 + i);
          if (2 * i >= lo && 2 * i < hi) to[2 * i] = t.x;
          if (2 * i + 1 >= lo && 2 * i + 1 < hi) to[2 * i + 1] = t.y;
        }
      } else {
#pragma unroll
        for (int h = 0; h < VEC / 4; ++h) {
          const float2 t = value(k * VEC / 2 + 2 * h), u = value(k * VEC / 2 + 2 * h + 1);
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
      for (int g = 0; g < groups; ++g) t += sums[g * a.D + c];
    }
    if (LAYER && a.db) {
      for (int g = 0; g < groups; ++g) u += sums[(groups + g) * a.D + c];
    }
    if (a.cluster) {  // only this thread reads or writes column c of this block
      sums[c] = t;
      if (LAYER) sums[groups * a.D + c] = u;
    } else {
      if (a.dw) a.part_w[row + c] = t;
      if (LAYER && a.db) a.part_b[row + c] = u;
    }
  }
  if (!a.cluster) return;
  // The grid is one cluster: the blocks share out the columns and add one
  // another's sums in the order of their ranks.
  cluster_sync();
  const uint32_t here = smem_u32(sums), ranks = gridDim.x;
  for (int c = static_cast<int>(blockIdx.x) * threads + tid; c < a.D; c += static_cast<int>(ranks) * threads) {
    float t = 0.0f, u = 0.0f;
    for (uint32_t r = 0; r < ranks; ++r) {
      const uint32_t other = mapa_shared(here, r);
      t += load_cluster(other + 4u * c);
      if (LAYER) u += load_cluster(other + 4u * (groups * a.D + c));
    }
    if (a.dw) store_param(a.dw, a.p_type, c, t);
    if (LAYER && a.db) store_param(a.db, a.p_type, c, u);
  }
  cluster_sync();  // no block leaves while another reads its sums
}

// Rows too long for the registers of one block: grad_x by one block per row in
// two passes over it, the parameter gradients column-wise by cols_kernel.  bf16
// 2,048 x 20,000: 99 us for a layer norm, 90 for an RMS norm; 2,048 x 20,001, by
// elements, 289 us.
template <typename TX, typename TY, int VEC, bool LAYER>
__global__ void __launch_bounds__(MAX_THREADS) bwd_long_kernel(NormBwd a) {
  __shared__ __align__(16) float sm[2][slots(MAX_THREADS)];
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
    xv.load_constant(x + c);
    gv.load_constant(dy + c);
    load_gain<LAYER, VEC, false, true>(a.w, a.p_type, a.offset, c, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float z = (xv.get(e) - mean) * rstd, g = gv.get(e) * w[e];
      if (LAYER) s.x += g;
      s.y += g * z;
    }
  }
  s = LAYER ? group_sum2(s, sm[0], slots(MAX_THREADS)) : make_float2(0.0f, group_sum(s.y, sm[0]));
  s.x *= inv_d;
  s.y *= inv_d;
#pragma unroll 2
  for (int64_t c = first; c < a.D; c += step) {
    Vec<TX, VEC> xv;
    Vec<TY, VEC> gv;
    float w[VEC], o[VEC];
    xv.load_constant(x + c);
    gv.load_constant(dy + c);
    load_gain<LAYER, VEC, false, true>(a.w, a.p_type, a.offset, c, w);
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
    xv.load_constant(static_cast<const TX*>(a.x) + a.xm.at(static_cast<int>(n)) + c);
    gv.load_constant(static_cast<const TY*>(a.dy) + a.gm.at(static_cast<int>(n)) + c);
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
// adds 32 columns: its warps take the parts w, w + WARPS, ... in order, LOADS of
// them in flight at once, and warp 0 adds the warps in order.  blockIdx.y = 0: the
// weight's, 1: the bias's.  Bound by latency, about 2 us behind the kernel that it
// follows; with the loads in a loop of five instead, 3.
template <int WARPS, int LOADS>
__global__ void __launch_bounds__(32 * WARPS) reduce_kernel(const float* part_w, const float* part_b, int parts, int D,
                                                            int p_type, void* dw, void* db) {
  __shared__ float ws[WARPS][32];
  wait_for_previous();
  void* out = blockIdx.y == 0 ? dw : db;
  if (!out) return;
  const float* part = blockIdx.y == 0 ? part_w : part_b;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < D) {
    for (int first = threadIdx.y; first < parts; first += WARPS * LOADS) {
      float v[LOADS];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int p = first + i * WARPS;
        v[i] = p < parts ? part[static_cast<int64_t>(p) * D + c] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i) s += v[i];
    }
  }
  ws[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    s = 0.0f;
    for (int i = 0; i < WARPS; ++i) s += ws[i][threadIdx.x];
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
  return launch_after(fwd_few_kernel<TX, TY, VEC, K, LAYER>, dim3(static_cast<unsigned>(a.N)),
                      dim3(group_threads(vecs, K)), 0, 1, s, a);
}

constexpr int MAX_SMEM = 227 * 1024 - 2048;   // dynamic shared memory of a block, beside what the kernels declare
constexpr int PLAIN_SMEM = 48 * 1024 - 2048;  // of a block that has not asked for more

// Vectors that a row may touch, and floats of its parameters in shared memory.
constexpr bool is_shifted(Access access) { return access == Access::SHIFTED || access == Access::REALIGNED; }
template <int VEC, Access A>
int64_t row_vecs(int64_t D) {
  return is_shifted(A) ? (D + 2 * VEC - 2) / VEC : D / VEC;
}
template <int VEC, Access A>
int64_t param_floats(int64_t D) {
  return is_shifted(A) ? VEC * row_vecs<VEC, A>(D) : D;
}

template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER, Access A>
cudaError_t run_fwd(const NormFwd& a, int tpr, cudaStream_t s) {
  auto kernel = fwd_kernel<TX, TY, VEC, K, KF, LAYER, A>;
  const int smem = static_cast<int>(sizeof(float) * param_floats<VEC, A>(a.D)) * (LAYER ? 2 : 1);
  // Two blocks of 256 threads an SM, where their parameters do not fit twice one of 512: with five to eight vectors of
  // 16-bit values a thread (120 to 128 registers) these fill the registers.  Fewer vectors (40 to 64 registers for one
  // to three of them) leave up to half of the registers idle, and groups of 96 threads some of the warps.
  const bool pair = 2 * (smem + 2048) <= MAX_SMEM;
  const int groups = std::max(1, (pair ? 256 : MAX_THREADS) / tpr);
  const int per_sm = std::max(1, MAX_THREADS / (tpr * groups));
  const int grid = static_cast<int>(std::min<int64_t>(cdiv(a.N, groups), a.sms * per_sm));
  if (smem > PLAIN_SMEM) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    if (e != cudaSuccess) return e;
  }
  return launch_after(kernel, dim3(grid), dim3(tpr, groups), smem, 1, s, a);
}

// Launches fwd_kernel for rows that the registers of one block hold; false for longer ones.
template <typename TX, typename TY, int VEC, bool LAYER, Access A>
bool fwd_in_registers(const NormFwd& a, cudaStream_t s, cudaError_t* e) {
  const int64_t vecs = row_vecs<VEC, A>(a.D);
  if (static_cast<int64_t>(sizeof(float)) * param_floats<VEC, A>(a.D) * (LAYER ? 2 : 1) > MAX_SMEM) return false;
  if constexpr (VEC > 1) {
    // Short rows with 4 vectors a thread: 65,536 x 256 15.2 us against 16.0 with 8; 1,024 wide 46.0 against 45.5.
    const int tpr = group_threads(vecs, vecs <= 64 ? 4 : 8);
    if (tpr > MAX_THREADS) return false;
    const int64_t each = cdiv(vecs, tpr);  // vectors a thread; all but its last are there in every thread
    if constexpr (!is_shifted(A)) {      // whose rows have columns enough for three
      if (each <= 2) {
        *e = each == 1 ? run_fwd<TX, TY, VEC, 1, 0, LAYER, A>(a, tpr, s) : run_fwd<TX, TY, VEC, 2, 1, LAYER, A>(a, tpr, s);
        return true;
      }
    }
    switch (each) {
      case 3: *e = run_fwd<TX, TY, VEC, 3, 2, LAYER, A>(a, tpr, s); break;
      case 4: *e = run_fwd<TX, TY, VEC, 4, 3, LAYER, A>(a, tpr, s); break;
      case 5: *e = run_fwd<TX, TY, VEC, 5, 4, LAYER, A>(a, tpr, s); break;
      case 6: *e = run_fwd<TX, TY, VEC, 6, 5, LAYER, A>(a, tpr, s); break;
      case 7: *e = run_fwd<TX, TY, VEC, 7, 6, LAYER, A>(a, tpr, s); break;
      default: *e = run_fwd<TX, TY, VEC, 8, 7, LAYER, A>(a, tpr, s); break;
    }
  } else {
    *e = run_fwd<TX, TY, VEC, 4, 0, LAYER, A>(a, group_threads(vecs, 4), s);
  }
  return true;
}

// A block per row while an SM has four rows or 16 KiB of them at most.  Measured
// on both sides (bf16 layer norm): 608 x 2,048 3.6 us against 3.9 by the
// persistent groups, 912 x 2,048 4.6 against 3.9; 304 x 4,096 3.6 against 4.5,
// 608 x 4,096 5.2 against 4.4.
template <typename TX, typename TY, int VEC, bool LAYER>
bool fwd_few(const NormFwd& a, cudaStream_t s, cudaError_t* e) {
  const int64_t vecs = a.D / VEC;
  if (a.N > 4 * a.sms || static_cast<int64_t>(sizeof(TX)) * a.N * a.D > int64_t(16384) * a.sms ||
      vecs > 4 * MAX_THREADS)
    return false;
  *e = vecs <= MAX_THREADS ? run_fwd_few<TX, TY, VEC, 1, LAYER>(a, vecs, s)
                           : run_fwd_few<TX, TY, VEC, 4, LAYER>(a, vecs, s);
  return true;
}

template <typename TX, typename TY, int VEC, bool LAYER>
cudaError_t fwd_long(const NormFwd& a, cudaStream_t s) {
  fwd_long_kernel<TX, TY, VEC, LAYER><<<static_cast<unsigned>(a.N), MAX_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TX, typename TY, bool LAYER>
cudaError_t fwd(const NormFwd& a, Access access, cudaStream_t s, int* launches) {
  constexpr int VEC = 16 / sizeof(TX);
  if (a.N == 0) return cudaSuccess;
  ++*launches;
  cudaError_t e = cudaSuccess;
  if (access == Access::WIDE) {
    if (fwd_few<TX, TY, VEC, LAYER>(a, s, &e) || fwd_in_registers<TX, TY, VEC, LAYER, Access::WIDE>(a, s, &e))
      return e;
    return fwd_long<TX, TY, VEC, LAYER>(a, s);
  }
  if (fwd_few<TX, TY, 1, LAYER>(a, s, &e)) return e;
  if (access == Access::SHIFTED     ? fwd_in_registers<TX, TY, VEC, LAYER, Access::SHIFTED>(a, s, &e)
      : access == Access::REALIGNED ? fwd_in_registers<TX, TY, VEC, LAYER, Access::REALIGNED>(a, s, &e)
                                    : fwd_in_registers<TX, TY, 1, LAYER, Access::SINGLE>(a, s, &e))
    return e;
  return fwd_long<TX, TY, 1, LAYER>(a, s);
}

constexpr int CLUSTER = 8;  // blocks, the portable limit
template <typename TX, typename TY, int VEC, int K, int KF, bool LAYER, Access A,
          int THREADS = bwd_threads<TX, VEC, K, LAYER>()>
cudaError_t run_bwd(const NormBwd& a, int tpr, int* parts, cudaStream_t s) {
  auto kernel = bwd_kernel<TX, TY, VEC, K, KF, LAYER, A, THREADS>;
  const int groups = std::max(1, THREADS / tpr);
  NormBwd b = a;
  // One row a group at most, of a quarter of the block's threads: one launch less, 1 x 896 4.5 us against 4.9 by two,
  // 300 x 128 5.2 against 5.8, 64 x 896 5.5 both; with two rows a group 7.2 against 5.4, with longer rows 7.9 against
  // 7.0 (16 x 4,096).
  b.cluster = (a.dw || a.db) && groups >= 4 && a.N <= static_cast<int64_t>(CLUSTER) * groups;
  // In multiples of 8 blocks, so that a group's rows are all shifted alike.
  int blocks = static_cast<int>(std::min<int64_t>(std::min(NORM_MAX_PARTS, std::max(8, a.sms / 8 * 8)),
                                                  cdiv(a.N, groups)));
  if (b.cluster) {
    int size = 1;
    while (size < blocks) size *= 2;
    blocks = size;
  }
  *parts = b.cluster ? 0 : blocks;
  const int64_t sums = static_cast<int64_t>(a.D) * groups * (LAYER && (is_shifted(A) || groups > 1) ? 2 : 1);
  const int64_t smem = std::max<int64_t>(
      sizeof(float) * sums, bwd_ring_bytes<TX, TY, VEC, K, THREADS>() + sizeof(float) * param_floats<VEC, A>(a.D));
  if (smem > PLAIN_SMEM) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
    if (e != cudaSuccess) return e;
  }
  return launch_after(kernel, dim3(blocks), dim3(tpr, groups), static_cast<size_t>(smem),
                      b.cluster ? static_cast<unsigned>(blocks) : 1u, s, b);
}

// Launches bwd_kernel for rows that the registers of one block hold; false for longer ones.
template <typename TX, typename TY, int VEC, bool LAYER, Access A>
bool bwd_in_registers(const NormBwd& a, int* parts, cudaStream_t s, cudaError_t* e) {
  const int64_t vecs = row_vecs<VEC, A>(a.D);
  if constexpr (VEC > 1) {
    constexpr int K = 16 / VEC;
    const int tpr = group_threads(vecs, K);
    if constexpr (LAYER && VEC == 8) {
      if (2 * tpr > MAX_THREADS && 2 * tpr <= WIDER) {
        *e = run_bwd<TX, TY, VEC, K, K - 1, LAYER, A, WIDER>(a, tpr, parts, s);
        return true;
      }
    }
    if (tpr <= bwd_threads<TX, VEC, K, LAYER>()) {
      const int64_t each = cdiv(vecs, tpr);  // vectors a thread; all but its last are there in every thread
      if constexpr (!is_shifted(A)) {      // whose rows have columns enough for more than half of K
        if (each <= K / 2) {
          *e = each == 1 ? run_bwd<TX, TY, VEC, 1, 0, LAYER, A>(a, tpr, parts, s)
                         : run_bwd<TX, TY, VEC, 2, 1, LAYER, A>(a, tpr, parts, s);
          return true;
        }
      }
      *e = each < K ? run_bwd<TX, TY, VEC, K / 2 + 1, K / 2, LAYER, A>(a, tpr, parts, s)
                    : run_bwd<TX, TY, VEC, K, K - 1, LAYER, A>(a, tpr, parts, s);
      return true;
    }
    if (vecs > 2 * K * MAX_THREADS) return false;
    // as few values a thread as 512 threads allow; blocks of more have taken all rows of up to 3 K / 2 vectors
    if constexpr (K * bwd_threads<TX, VEC, K, LAYER>() < 3 * K / 2 * MAX_THREADS) {
      if (vecs <= 3 * K / 2 * MAX_THREADS) {
        *e = run_bwd<TX, TY, VEC, 3 * K / 2, K - 1, LAYER, A>(a, group_threads(vecs, 3 * K / 2), parts, s);
        return true;
      }
    }
    *e = run_bwd<TX, TY, VEC, 2 * K, 3 * K / 2 - 1, LAYER, A>(a, group_threads(vecs, 2 * K), parts, s);
  } else {
    *e = run_bwd<TX, TY, VEC, 4, 0, LAYER, A>(a, group_threads(vecs, 4), parts, s);
  }
  return true;
}

template <typename TX, typename TY, int VEC, bool LAYER>
cudaError_t bwd_long(const NormBwd& a, int* parts, cudaStream_t s, int* launches) {
  if (a.dx) bwd_long_kernel<TX, TY, VEC, LAYER><<<static_cast<unsigned>(a.N), MAX_THREADS, 0, s>>>(a);
  if (a.dw || a.db) {
    const int64_t tiles = cdiv(a.D / VEC, 128);
    *parts =
        static_cast<int>(std::min<int64_t>({NORM_MAX_PARTS, cdiv(a.N, 8), std::max<int64_t>(1, 8 * a.sms / tiles)}));
    *launches += a.dx ? 1 : 0;
    cols_kernel<TX, TY, VEC, LAYER>
        <<<dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(*parts)), 128, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename TX, typename TY, bool LAYER>
cudaError_t bwd(const NormBwd& a, Access access, cudaStream_t s, int* launches) {
  constexpr int VEC = 16 / sizeof(TX);
  int parts = 0;
  if (a.N > 0 && (a.dx || a.dw || a.db)) {
    ++*launches;
    cudaError_t e = cudaSuccess;
    if (access == Access::WIDE) {
      if (!bwd_in_registers<TX, TY, VEC, LAYER, Access::WIDE>(a, &parts, s, &e))
        e = bwd_long<TX, TY, VEC, LAYER>(a, &parts, s, launches);
    } else if (!(access == Access::SHIFTED     ? bwd_in_registers<TX, TY, VEC, LAYER, Access::SHIFTED>(a, &parts, s, &e)
                 : access == Access::REALIGNED ? bwd_in_registers<TX, TY, VEC, LAYER, Access::REALIGNED>(a, &parts, s, &e)
                                               : bwd_in_registers<TX, TY, 1, LAYER, Access::SINGLE>(a, &parts, s, &e))) {
      e = bwd_long<TX, TY, 1, LAYER>(a, &parts, s, launches);
    }
    if (e != cudaSuccess) return e;
  }
  if ((!a.dw && !a.db) || (a.N > 0 && parts == 0)) return cudaSuccess;  // parts == 0: the cluster has written them
  ++*launches;
  const dim3 grid(static_cast<unsigned>(cdiv(a.D, 32)), LAYER ? 2 : 1);
  // Both hold the 152 parts of a full grid at once.  Few warps start sooner, where an SM has one block of them: layer
  // norm of 9,360 x 896 15.1 us and 16.2 with 16 warps, 3,640 x 2,304 16.1 and 16.9, but 2,048 x 4,096, 256 blocks,
  // 18.3 and 17.2; 8,376 x 1,001, behind the longer end of a kernel of shifted rows, 22.3 and 21.3.
  if (static_cast<int64_t>(grid.x) * grid.y <= a.sms && a.D % 8 == 0) {
    return launch_after(reduce_kernel<8, 20>, grid, dim3(32, 8), 0, 1, s, a.part_w, a.part_b, parts, a.D, a.p_type,
                        a.dw, a.db);
  }
  return launch_after(reduce_kernel<16, 10>, grid, dim3(32, 16), 0, 1, s, a.part_w, a.part_b, parts, a.D, a.p_type,
                      a.dw, a.db);
}

}  // namespace norm
}  // namespace cce

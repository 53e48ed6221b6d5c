// Global gradient norm and clipping over many tensors (include/cce_ops.h).
//
//   norm = sqrt(sum x^2) or max |x| over all elements;  out = x * min(1, max_norm / (norm + eps))
//
// Bound by memory: every element is read once for the norm and, unless the
// factor is 1 in place, read again and written.  The tensors are cut into
// chunks, which the blocks of one launch take in turn, so that a launch covers
// hundreds of tensors of any size; the table of tensors travels in the kernel's
// parameters (no copy to the device, nothing to keep alive for a captured
// graph).  The second pass walks the chunks backwards: what the first pass read
// last is still in L2.
//
// Measured: the norm of an 805 MB bf16 tensor 114 us (7.1 TB/s); 444 M bf16
// gradients in 291 tensors clipped into fp32, 888 MB read twice and 1.8 GB
// written, 558 us (6.4 TB/s); 0.5 M values 5.2 us for both launches, all latency.
//
// A thread sums the squares of up to 64 values in fp32; from there on a sum is a
// pair of fp32 values, the rounded sum and what the roundings lost, up to the
// norm itself.  fp64 adds are slow on a GB300: with them 14.7 M bf16 values were
// clipped into fp32 in 27 us and not 18.  Where a block's sum overflows, or is so
// small that squares may have underflowed, the block goes over its values again
// in fp64.  Every order is fixed.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>

#include "elements.cuh"
#include "internal.h"

namespace cce {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 8;                  // 16-byte loads in flight per thread
constexpr int ROUND = THREADS * UNROLL * 8;  // elements of one unrolled round of 16-bit values
// 152 SMs x 4 resident blocks: 2 an SM clip the 444 M values in 590 us, 3 in 579, 4 in 567.
constexpr int GRID = 608;
constexpr int MAX_TENSORS = 1000;          // per launch: what 32 KB of parameters hold
constexpr int FEW_TENSORS = 32;            // a launch with 1 KB of them
// Of one tensor: then the chunks of MAX_TENSORS of them can be counted in 32 bits.
constexpr int64_t MAX_ELEMENTS = int64_t(1) << 35;
static_assert(MAX_ELEMENTS / ROUND * MAX_TENSORS < int64_t(1) << 32, "chunk numbers");

struct Tensor {
  const void* in;
  void* out;
  int64_t n;
  uint32_t first_chunk;
  uint8_t in_type, out_type, wide_in, wide_both;
};
static_assert(sizeof(Tensor) == 32, "table entry");

template <int M>
struct Batch {
  Tensor t[M];
  int count;
  int chunk;  // elements
  uint32_t chunks;
  int in_place;  // every output is its input
};
static_assert(sizeof(Batch<MAX_TENSORS>) <= 32000 + 64, "kernel parameters");

// A block's part of the norm: the sum of squares as hi + lo, or, where hi is
// infinite, as `wide`; or the largest magnitude as hi.
struct Part {
  float hi, lo;
  double wide;
};

struct Clip {
  const Part* part;
  int parts;
  int norm_type;
  float max_norm, eps;
  float* norm;  // written by block 0, may be null
};

// The last tensor whose first chunk is <= chunk.
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

// Larger of two magnitudes; NaN wins.
__device__ __forceinline__ float larger(float a, float b) { return b > a || b != b ? b : a; }

// A sum of fp32 values with what its roundings lost (Knuth's exact two-term sum).
struct Sum {
  float hi = 0.0f, lo = 0.0f;

  __device__ __forceinline__ void add(float v, float low = 0.0f) {
    const float t = hi + v, part = t - hi;
    lo += ((hi - (t - part)) + (v - part)) + low;
    hi = t;
  }
};

// Over the block, in a fixed order; the result is thread 0's.
__device__ Sum block_sum(Sum v, bool inf) {
  __shared__ float2 sm[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_down_sync(0xffffffffu, v.hi, o), lo = __shfl_down_sync(0xffffffffu, v.lo, o);
    if (inf) {
      v.hi = larger(v.hi, hi);
    } else {
      v.add(hi, lo);
    }
  }
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_float2(v.hi, v.lo);
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) {
      if (inf) {
        v.hi = larger(v.hi, sm[w].x);
      } else {
        v.add(sm[w].x, sm[w].y);
      }
    }
  }
  return v;
}

__device__ double block_sum64(double v) {
  __shared__ double sm[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_down_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < THREADS / 32; ++w) v += sm[w];
  }
  return v;
}

// What a thread gathers: squares or the largest magnitude.
struct Gather {
  Sum sum;            // of the rounds that have ended
  float s = 0.0f;     // of this round: sum of squares; or the largest magnitude
  uint32_t any = 0u;  // bits of the values but the signs

  template <typename T, int VEC>
  __device__ __forceinline__ void add(const Vec<T, VEC>& v, bool inf) {
    if (inf) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s = larger(s, fabsf(v.get(e)));
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float f = v.get(e);
        s += f * f;
      }
#pragma unroll
      for (int i = 0; i < Vec<T, VEC>::WORDS; ++i) any |= v.w[i] & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu);
    }
  }
  __device__ __forceinline__ void end_round(bool inf) {
    if (inf) return;
    sum.add(s);
    s = 0.0f;
  }
};

// The block's part of the norm.  Fewer than 2^31 squares lose less than 2^-119 to
// underflow, which is nothing beside a sum of 2^-80; below that, and where fp32
// overflows, `again` returns the sum of the thread's squares in fp64.
template <typename Again>
__device__ __forceinline__ void put_part(const Gather& g, bool inf, Part* part, Again again) {
  Sum v = g.sum;
  if (inf) v.hi = g.s;
  v = block_sum(v, inf);
  Part p{v.hi, v.lo, 0.0};
  const bool fits = inf || (v.hi >= 0x1p-80f && v.hi <= 3.0e38f);
  if (__syncthreads_or(threadIdx.x == 0 && !fits) && __syncthreads_or(g.any != 0u)) {
    p.wide = block_sum64(again());
    p.hi = INFINITY;
  }
  if (threadIdx.x == 0) part[blockIdx.x] = p;
}

// Rounds of U vectors a thread from vector v on, while whole rounds are left.
template <int U, typename T, int VEC>
__device__ __forceinline__ void gather_rounds(const T* p, int vecs, int& v, bool inf, Gather& g) {
#pragma unroll 1
  for (; v + THREADS * (U - 1) < vecs; v += THREADS * U) {
    Vec<T, VEC> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(p + static_cast<int64_t>(v + u * THREADS) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u) g.add(x[u], inf);
    g.end_round(inf);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void gather_chunk(const T* p, int n, bool inf, Gather& g) {
  const int vecs = n / VEC;
  int v = threadIdx.x;
  gather_rounds<UNROLL, T, VEC>(p, vecs, v, inf, g);
  gather_rounds<2, T, VEC>(p, vecs, v, inf, g);
  gather_rounds<1, T, VEC>(p, vecs, v, inf, g);
  if constexpr (VEC > 1) {
    const int i = vecs * VEC + threadIdx.x;
    if (i < n) {
      Vec<T, 1> x[1];
      x[0].load(p + i);
      g.add(x[0], inf);
      g.end_round(inf);
    }
  }
}

template <typename T>
__device__ __forceinline__ void gather_typed(const void* in, int64_t off, int n, bool wide, bool inf, Gather& g) {
  const T* p = static_cast<const T*>(in) + off;
  if (wide) {
    gather_chunk<T, 16 / sizeof(T)>(p, n, inf, g);
  } else {
    gather_chunk<T, 1>(p, n, inf, g);
  }
}

__device__ __forceinline__ float load_any(const void* p, int type, int64_t i) {
  if (type == CCE_F32) return static_cast<const float*>(p)[i];
  if (type == CCE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

template <int M>
__global__ void __launch_bounds__(THREADS, 4) norm_kernel(const __grid_constant__ Batch<M> b, int norm_type,
                                                       Part* part) {
  const bool inf = norm_type == CCE_NORM_INF;
  let_next_start();
  wait_for_previous();
  Gather g;
  for (uint32_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, c)];
    const int64_t off = static_cast<int64_t>(c - t.first_chunk) * b.chunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(b.chunk), t.n - off));
    if (t.in_type == CCE_F32) {
      gather_typed<float>(t.in, off, n, t.wide_in, inf, g);
    } else if (t.in_type == CCE_BF16) {
      gather_typed<__nv_bfloat16>(t.in, off, n, t.wide_in, inf, g);
    } else {
      gather_typed<__half>(t.in, off, n, t.wide_in, inf, g);
    }
  }
  put_part(g, inf, part, [&] {
    double wide = 0.0;
    for (uint32_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
      const Tensor& t = b.t[find_tensor(b, c)];
      const int64_t off = static_cast<int64_t>(c - t.first_chunk) * b.chunk;
      const int64_t end = min(off + b.chunk, t.n);
      for (int64_t i = off + threadIdx.x; i < end; i += THREADS) {
        const double f = load_any(t.in, t.in_type, i);
        wide += f * f;
      }
    }
    return wide;
  });
}

// Thread 0's result.
__device__ float wide_norm(const Part* part, int parts) {
  double t = 0.0;
  for (int i = threadIdx.x; i < parts; i += THREADS) {
    const Part p = part[i];
    t += p.hi < INFINITY ? static_cast<double>(p.hi) + static_cast<double>(p.lo) : p.wide;
  }
  return static_cast<float>(sqrt(block_sum64(t)));
}

// The norm from the block partials: every block computes it, in the same order.
__device__ float total_norm(const Clip& k) {
  __shared__ float result;
  wait_for_previous();
  const bool inf = k.norm_type == CCE_NORM_INF;
  Sum v;
  for (int i = threadIdx.x; i < k.parts; i += THREADS) {
    const float2 p = *reinterpret_cast<const float2*>(k.part + i);
    if (inf) {
      v.hi = larger(v.hi, p.x);
    } else {
      v.add(p.x, p.y);
    }
  }
  v = block_sum(v, inf);
  if (threadIdx.x == 0) result = inf ? v.hi : v.hi + v.lo <= 3.0e38f ? sqrtf(v.hi + v.lo) : INFINITY;
  __syncthreads();
  if (!inf && !(result < INFINITY)) {  // a block's part or the total is outside fp32's range
    const float wide = wide_norm(k.part, k.parts);
    if (threadIdx.x == 0) result = wide;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && k.norm) *k.norm = result;
  return result;
}

__global__ void __launch_bounds__(THREADS) finish_kernel(Clip k) { total_norm(k); }

// NaN for a NaN norm.  Where the quotient of two other values would be one, an infinite norm below an infinite limit or
// 0 by 0, nothing is clipped.
__device__ __forceinline__ float clip_factor(const Clip& k, float norm) {
  const float f = k.max_norm / (norm + k.eps);
  return f < 1.0f || norm != norm ? f : 1.0f;
}

template <typename TI, typename TO, int VEC>
__device__ __forceinline__ void scale_vec(const Vec<TI, VEC>& x, TO* q, float f) {
  float o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = x.get(e) * f;
  Vec<TO, VEC> y;
  y.set(o);
  y.store(q);
}

template <int U, typename TI, typename TO, int VEC>
__device__ __forceinline__ void scale_rounds(const TI* p, TO* q, int vecs, int& v, float f) {
#pragma unroll 1
  for (; v + THREADS * (U - 1) < vecs; v += THREADS * U) {
    Vec<TI, VEC> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(p + static_cast<int64_t>(v + u * THREADS) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u) scale_vec<TI, TO, VEC>(x[u], q + static_cast<int64_t>(v + u * THREADS) * VEC, f);
  }
}

template <typename TI, typename TO, int VEC>
__device__ __forceinline__ void scale_chunk(const TI* p, TO* q, int n, float f) {
  const int vecs = n / VEC;
  int v = threadIdx.x;
  scale_rounds<UNROLL, TI, TO, VEC>(p, q, vecs, v, f);
  scale_rounds<2, TI, TO, VEC>(p, q, vecs, v, f);
  scale_rounds<1, TI, TO, VEC>(p, q, vecs, v, f);
  if constexpr (VEC > 1) {
    const int i = vecs * VEC + threadIdx.x;
    if (i < n) {
      Vec<TI, 1> x;
      x.load(p + i);
      scale_vec<TI, TO, 1>(x, q + i, f);
    }
  }
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_typed(const Tensor& t, int64_t off, int n, float f) {
  const TI* p = static_cast<const TI*>(t.in) + off;
  TO* q = static_cast<TO*>(t.out) + off;
  if (t.wide_both) {  // neither access wider than 16 bytes, so that both are on consecutive addresses
    scale_chunk<TI, TO, 16 / (sizeof(TI) > sizeof(TO) ? sizeof(TI) : sizeof(TO))>(p, q, n, f);
  } else {
    scale_chunk<TI, TO, 1>(p, q, n, f);
  }
}

template <typename TI>
__device__ __forceinline__ void scale_from(const Tensor& t, int64_t off, int n, float f) {
  if (t.out_type == CCE_F32) {
    scale_typed<TI, float>(t, off, n, f);
  } else if (t.out_type == CCE_BF16) {
    scale_typed<TI, __nv_bfloat16>(t, off, n, f);
  } else {
    scale_typed<TI, __half>(t, off, n, f);
  }
}

template <int M>
__global__ void __launch_bounds__(THREADS, 4) scale_kernel(const __grid_constant__ Batch<M> b, Clip k) {
  const float f = clip_factor(k, total_norm(k));
  if (f == 1.0f && b.in_place) return;
  for (uint32_t i = blockIdx.x; i < b.chunks; i += gridDim.x) {
    const uint32_t c = b.chunks - 1 - i;
    const Tensor& t = b.t[find_tensor(b, c)];
    if (f == 1.0f && t.in == t.out) continue;
    const int64_t off = static_cast<int64_t>(c - t.first_chunk) * b.chunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(b.chunk), t.n - off));
    if (t.in_type == CCE_F32) {
      scale_from<float>(t, off, n, f);
    } else if (t.in_type == CCE_BF16) {
      scale_from<__nv_bfloat16>(t, off, n, f);
    } else {
      scale_from<__half>(t, off, n, f);
    }
  }
}

// ---------------------------------------------------------- strided tensors
__device__ __forceinline__ void strided_offsets(const cce_strided& t, int64_t i, int64_t* in, int64_t* out) {
  int64_t a = 0, b = 0;
#pragma unroll
  for (int d = 3; d > 0; --d) {
    const int64_t q = i / t.size[d], r = i - q * t.size[d];
    a += r * t.in_stride[d];
    b += r * t.out_stride[d];
    i = q;
  }
  *in = a + i * t.in_stride[0];
  *out = b + i * t.out_stride[0];
}

// One element at a time: few tensors take this path.  The left half of the columns of 8,192 x 4,096 bf16 values, 33 MB:
// from L2: norm 99 us, clipped into bf16 207; as one block of memory 7 and 14.
__global__ void __launch_bounds__(THREADS) strided_norm_kernel(const __grid_constant__ cce_strided t, int64_t n,
                                                               int norm_type, Part* part) {
  const bool inf = norm_type == CCE_NORM_INF;
  const int64_t first = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * THREADS;
  Gather g;
  for (int64_t i = first; i < n; i += step) {
    int64_t a, b;
    strided_offsets(t, i, &a, &b);
    Vec<float, 1> x;
    x.w[0] = __float_as_uint(load_any(t.in, t.in_type, a));
    g.add(x, inf);
    g.end_round(inf);
  }
  put_part(g, inf, part, [&] {
    double wide = 0.0;
    for (int64_t i = first; i < n; i += step) {
      int64_t a, b;
      strided_offsets(t, i, &a, &b);
      const double f = load_any(t.in, t.in_type, a);
      wide += f * f;
    }
    return wide;
  });
}

__global__ void __launch_bounds__(THREADS) strided_scale_kernel(const __grid_constant__ cce_strided t, int64_t n,
                                                                Clip k) {
  const float f = clip_factor(k, total_norm(k));
  if (f == 1.0f && t.in == t.out) return;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(THREADS) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * THREADS) {
    int64_t a, b;
    strided_offsets(t, i, &a, &b);
    store_param(t.out, t.out_type, b, load_any(t.in, t.in_type, a) * f);
  }
}

// --------------------------------------------------------------------- host
int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t type_bytes(int t) { return t == CCE_F32 ? 4 : 2; }
bool type_ok(int t) { return t == CCE_F32 || t == CCE_F16 || t == CCE_BF16; }
bool multiple(const void* p, int64_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0;
}

struct Row {
  const void* in;
  void* out;
  int64_t n;
  int in_type, out_type;
};

Row table_row(const int64_t* dense, int64_t i) {
  const int64_t* r = dense + 4 * i;
  return Row{reinterpret_cast<const void*>(r[0]), reinterpret_cast<void*>(r[1]), r[2], static_cast<int>(r[3] & 255),
             static_cast<int>(r[3] >> 8)};
}

int64_t elements(const cce_strided& t) { return t.size[0] * t.size[1] * t.size[2] * t.size[3]; }

cce_status check_tables(const int64_t* dense, int64_t n_dense, const cce_strided* strided, int64_t n_strided,
                        bool outputs) {
  if (n_dense < 0 || n_strided < 0) return CCE_ERR_SHAPE;
  if ((n_dense > 0 && !dense) || (n_strided > 0 && !strided)) return CCE_ERR_NULL;
  for (int64_t i = 0; i < n_dense; ++i) {
    const Row r = table_row(dense, i);
    if (!type_ok(r.in_type) || (outputs && !type_ok(r.out_type))) return CCE_ERR_ARG;
    if (r.n < 0 || r.n >= MAX_ELEMENTS) return CCE_ERR_SHAPE;
    if (r.n == 0) continue;
    if (!r.in || (outputs && !r.out)) return CCE_ERR_NULL;
    if (!multiple(r.in, type_bytes(r.in_type)) || (outputs && !multiple(r.out, type_bytes(r.out_type))))
      return CCE_ERR_ALIGN;
    if (outputs && r.in == r.out && r.in_type != r.out_type) return CCE_ERR_ARG;
  }
  for (int64_t i = 0; i < n_strided; ++i) {
    const cce_strided& t = strided[i];
    if (!type_ok(t.in_type) || (outputs && !type_ok(t.out_type))) return CCE_ERR_ARG;
    int64_t n = 1;
    for (int d = 0; d < 4; ++d) {
      if (t.size[d] < 0 || t.size[d] >= MAX_ELEMENTS || t.in_stride[d] < 0 || t.out_stride[d] < 0)
        return CCE_ERR_SHAPE;
      if (n > 0 && t.size[d] > MAX_ELEMENTS / n) return CCE_ERR_SHAPE;
      n *= t.size[d];
    }
    if (n == 0) continue;
    if (!t.in || (outputs && !t.out)) return CCE_ERR_NULL;
    if (!multiple(t.in, type_bytes(t.in_type)) || (outputs && !multiple(t.out, type_bytes(t.out_type))))
      return CCE_ERR_ALIGN;
    if (outputs && t.in == t.out) {
      if (t.in_type != t.out_type) return CCE_ERR_ARG;
      for (int d = 0; d < 4; ++d) {  // otherwise ordered: threads would write what others have yet to read
        if (t.size[d] > 1 && t.in_stride[d] != t.out_stride[d]) return CCE_ERR_ARG;
      }
    }
  }
  return CCE_OK;
}

// An output block that overlaps another block would be read and written in any
// order by the blocks of one launch.
struct Span {
  uintptr_t lo, hi;
  bool out;
};

cce_status check_overlap(const int64_t* dense, int64_t n_dense) {
  Span* spans = new (std::nothrow) Span[2 * static_cast<size_t>(std::max<int64_t>(1, n_dense))];
  if (!spans) return CCE_ERR_CUDA;
  int64_t m = 0;
  for (int64_t i = 0; i < n_dense; ++i) {
    const Row r = table_row(dense, i);
    if (r.n == 0) continue;
    const uintptr_t in = reinterpret_cast<uintptr_t>(r.in), out = reinterpret_cast<uintptr_t>(r.out);
    if (in != out) spans[m++] = Span{in, in + static_cast<uintptr_t>(r.n * type_bytes(r.in_type)), false};
    spans[m++] = Span{out, out + static_cast<uintptr_t>(r.n * type_bytes(r.out_type)), true};
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

// Fills `b` with tensors from *next on; what does not fit waits for the next batch.
template <int M>
void fill_batch(Batch<M>& b, const int64_t* dense, int64_t n_dense, int chunk, int64_t* next) {
  b.count = 0;
  b.chunk = chunk;
  b.in_place = 1;
  int64_t chunks = 0;
  for (; *next < n_dense && b.count < M; ++*next) {
    const Row r = table_row(dense, *next);
    if (r.n == 0) continue;
    const int64_t vec = 16 / type_bytes(r.in_type);
    Tensor& t = b.t[b.count++];
    t.in = r.in;
    t.out = r.out;
    t.n = r.n;
    t.first_chunk = static_cast<uint32_t>(chunks);
    if (r.in != r.out) b.in_place = 0;
    t.in_type = static_cast<uint8_t>(r.in_type);
    t.out_type = static_cast<uint8_t>(r.out_type);
    t.wide_in = multiple(r.in, 16);
    t.wide_both = t.wide_in && multiple(r.out, std::min<int64_t>(16, vec * type_bytes(r.out_type)));
    chunks += cdiv64(r.n, chunk);
  }
  b.chunks = static_cast<uint32_t>(chunks);
}

int grid_of(uint32_t chunks) { return static_cast<int>(std::min<uint32_t>(GRID, chunks)); }

// Elements of a chunk: one unrolled round of 16-bit values, but
// - a quarter of it where that leaves half of the blocks without work: 0.5 M bf16
//   values are clipped into fp32 in 5.2 us and not 5.7, 1 M in 5.2 and not 5.8;
//   2 M, where it would fill the grid, take 6.7 us so and 6.2 in whole rounds;
// - four rounds where every block still has four such chunks: 305 M values take
//   395 us and not 397, 287 and not 290 into bf16.
int chunk_of(int64_t total) {
  if (total <= int64_t(GRID / 2) * (ROUND / 4)) return ROUND / 4;
  return total >= int64_t(16) * GRID * ROUND ? 4 * ROUND : ROUND;
}

// The norm pass (clip null) or the scaling pass over the dense tensors.
template <int M>
cudaError_t run_dense(const int64_t* dense, int64_t n_dense, int chunk, int norm_type, const Clip* clip, Part* part,
                      int* parts, cudaStream_t s, int* launches) {
  Batch<M> b;
  for (int64_t next = 0; next < n_dense;) {
    fill_batch(b, dense, n_dense, chunk, &next);
    if (b.count == 0) continue;
    const int grid = grid_of(b.chunks);
    if (clip) {
      const cudaError_t e = launch_after(scale_kernel<M>, dim3(grid), dim3(THREADS), 0, 1, s, b, *clip);
      if (e != cudaSuccess) return e;
    } else {
      const cudaError_t e =
          launch_after(norm_kernel<M>, dim3(grid), dim3(THREADS), 0, 1, s, b, norm_type, part + *parts);
      if (e != cudaSuccess) return e;
      *parts += grid;
    }
    ++*launches;
  }
  return cudaSuccess;
}

cudaError_t pass(const int64_t* dense, int64_t n_dense, const cce_strided* strided, int64_t n_strided, int norm_type,
                 const Clip* clip, Part* part, int* parts, cudaStream_t s, int* launches) {
  int64_t total = 0;
  for (int64_t i = 0; i < n_dense; ++i) total += dense[4 * i + 2];
  const int chunk = chunk_of(total);
  cudaError_t e = n_dense <= FEW_TENSORS
                      ? run_dense<FEW_TENSORS>(dense, n_dense, chunk, norm_type, clip, part, parts, s, launches)
                      : run_dense<MAX_TENSORS>(dense, n_dense, chunk, norm_type, clip, part, parts, s, launches);
  for (int64_t i = 0; i < n_strided && e == cudaSuccess; ++i) {
    const int64_t n = elements(strided[i]);
    if (n == 0) continue;
    const int grid = static_cast<int>(std::min<int64_t>(GRID, cdiv64(n, THREADS)));
    if (clip) {
      strided_scale_kernel<<<grid, THREADS, 0, s>>>(strided[i], n, *clip);
    } else {
      strided_norm_kernel<<<grid, THREADS, 0, s>>>(strided[i], n, norm_type, part + *parts);
      *parts += grid;
    }
    ++*launches;
    e = cudaGetLastError();
  }
  return e;
}

size_t workspace_bytes(int64_t n_dense, int64_t n_strided) {
  const int64_t launches = std::max<int64_t>(1, cdiv64(n_dense, MAX_TENSORS)) + n_strided;
  return sizeof(Part) * GRID * static_cast<size_t>(launches);
}

cce_status run(const int64_t* dense, int64_t n_dense, const cce_strided* strided, int64_t n_strided, int norm_type,
               bool clipping, float max_norm, float eps, float* norm, void* workspace, size_t ws_bytes,
               void* stream) {
  if (norm_type != CCE_NORM_INF && norm_type != CCE_NORM_2) return CCE_ERR_ARG;
  if (clipping && (!(max_norm >= 0.0f) || !std::isfinite(eps) || eps < 0.0f)) return CCE_ERR_ARG;
  cce_status st = check_tables(dense, n_dense, strided, n_strided, clipping);
  if (st != CCE_OK) return st;
  if (!norm || !workspace) return CCE_ERR_NULL;
  if (!multiple(norm, 4) || !multiple(workspace, 16)) return CCE_ERR_ALIGN;
  if (ws_bytes < workspace_bytes(n_dense, n_strided)) return CCE_ERR_WORKSPACE;
  if (clipping) {
    st = check_overlap(dense, n_dense);
    if (st != CCE_OK) return st;
  }
  int sms = 0;
  st = static_cast<cce_status>(device_ready(&sms));
  if (st != CCE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Part* part = static_cast<Part*>(workspace);
  int parts = 0, launches = 0;
  cudaError_t e = pass(dense, n_dense, strided, n_strided, norm_type, nullptr, part, &parts, s, &launches);
  const Clip k{part, parts, norm_type, max_norm, eps, norm};
  if (e == cudaSuccess && clipping && parts > 0)
    e = pass(dense, n_dense, strided, n_strided, norm_type, &k, part, &parts, s, &launches);
  if (e == cudaSuccess && (!clipping || parts == 0)) {
    e = launch_after(finish_kernel, dim3(1), dim3(THREADS), 0, 1, s, k);
    ++launches;
  }
  count_launches(launches);
  return e == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

}  // namespace
}  // namespace cce

using namespace cce;

extern "C" {

size_t cce_grad_norm_workspace_bytes(int64_t n_dense, int64_t n_strided) {
  return n_dense < 0 || n_strided < 0 ? 0 : workspace_bytes(n_dense, n_strided);
}

cce_status cce_grad_norm(const int64_t* dense, int64_t n_dense, const cce_strided* strided, int64_t n_strided,
                         int norm_type, float* norm, void* workspace, size_t ws_bytes, void* stream) {
  return run(dense, n_dense, strided, n_strided, norm_type, false, 0.0f, 0.0f, norm, workspace, ws_bytes, stream);
}

cce_status cce_clip_grads(const int64_t* dense, int64_t n_dense, const cce_strided* strided, int64_t n_strided,
                          int norm_type, float max_norm, float eps, float* norm, void* workspace, size_t ws_bytes,
                          void* stream) {
  return run(dense, n_dense, strided, n_strided, norm_type, true, max_norm, eps, norm, workspace, ws_bytes, stream);
}

}  // extern "C"

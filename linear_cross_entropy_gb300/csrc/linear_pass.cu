// Element-wise passes of the layers in front of the head, all bound by memory:
//
//   join  the epilogue over the partial sums of a product whose K was split
//   grad  dz = dy f'(z), or of a gated layer dgate = dy u f'(g) and dup = dy f(g),
//         in the type of the products that follow, and the sums of dz over the rows
//   copy  rows that are off 16 bytes or at two pitches into ones that the products take
//
// The vectors are of 16 bytes (fp32 ones of partial sums too) where all rows start on
// them.  A gated layer's grad of 4,096 x 4,864 takes some 35 us for 200 MB.
#include <algorithm>

#include "internal.h"
#include "linear.h"
#include "linear_epilogue.cuh"

namespace cce {
namespace {

constexpr int THREADS = 256;
constexpr int JOIN_COLS = 64;  // vectors of a row that a block works on, of THREADS / JOIN_COLS rows

template <typename T, bool GATED, int VEC>
__global__ void __launch_bounds__(THREADS) join_kernel(const float* part, int I, int J, int splits, LinEpilogue e) {
  let_next_start();
  wait_for_previous();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * JOIN_COLS + threadIdx.x % JOIN_COLS) * VEC;
  if (i >= I) return;
  const int64_t size = static_cast<int64_t>(I) * J, rows = static_cast<int64_t>(gridDim.y) * (THREADS / JOIN_COLS);
  for (int64_t j = static_cast<int64_t>(blockIdx.y) * (THREADS / JOIN_COLS) + threadIdx.x / JOIN_COLS; j < J; j += rows) {
    float z0[VEC] = {}, z1[VEC] = {};
    const float* p = part + j * I + i;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {  // in order
      Vec<float, VEC> v, u;
      v.load(p);
      p += size;
      if (GATED) {
        u.load(p);
        p += size;
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        z0[k] += v.get(k);
        if (GATED) z1[k] += u.get(k);
      }
    }
    finish_row<T, GATED>(e, j, i, z0, z1);
  }
}

// ------------------------------------------------------------------- backward
constexpr int COLS = 32, GROUPS = THREADS / COLS;  // a block: vectors of a row, rows at a time
// Rows of a thread in flight, of three blocks an SM: with four rows and the one block that their registers leave in a gated
// layer, 4,096 x 4,864 from L2 and memory took 5 us longer.
constexpr int UNROLL = 2;

template <int ACT, bool GATED, int VEC>
__device__ __forceinline__ void grad_as(float (&d0)[VEC], float (&d1)[VEC], const float (&dy)[VEC],
                                        const float (&z0)[VEC], const float (&z1)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float2 f = activate_both<ACT>(z0[e]);
    if (GATED) {
      d0[e] = dy[e] * z1[e] * f.y;
      d1[e] = dy[e] * f.x;
    } else {
      d0[e] = dy[e] * f.y;
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void set_part(uint32_t* w, const float (&f)[VEC]) {
  Vec<T, VEC> v;
  v.set(f);
#pragma unroll
  for (int x = 0; x < (VEC + 1) / 2; ++x) w[x] = v.w[x];
}

template <typename T, typename TY, bool GATED, int VEC>
__global__ void __launch_bounds__(THREADS, 3) grad_kernel(const __grid_constant__ LinGrad a) {
  let_next_start();
  wait_for_previous();
  const int tx = static_cast<int>(threadIdx.x) % COLS, ty = static_cast<int>(threadIdx.x) / COLS;
  const int col = (static_cast<int>(blockIdx.x) * COLS + tx) * VEC;
  constexpr int PART = VEC < 4 ? VEC : 4;  // values at a time, for fewer registers
  float sum[VEC] = {};
  if (col < a.N) {
    const int64_t step = static_cast<int64_t>(gridDim.y) * GROUPS;
    for (int64_t r0 = static_cast<int64_t>(blockIdx.y) * GROUPS + ty; r0 < a.M; r0 += step * UNROLL) {
      Vec<TY, VEC> dy[UNROLL];
      Vec<T, VEC> z0[UNROLL], z1[UNROLL];
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int64_t r = r0 + u * step;
        if (r < a.M) {
          dy[u].load(static_cast<const TY*>(a.dy) + r * a.dy_pitch + col);
          if (a.act != CCE_ACT_NONE || GATED) z0[u].load(static_cast<const T*>(a.z[0]) + r * a.z_pitch[0] + col);
          if (GATED) z1[u].load(static_cast<const T*>(a.z[1]) + r * a.z_pitch[1] + col);
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) {
        const int64_t r = r0 + u * step;
        if (r >= a.M) break;
        Vec<T, VEC> o0, o1;
#pragma unroll
        for (int h = 0; h < VEC; h += PART) {
          float g[PART], f0[PART], f1[PART], d0[PART], d1[PART];
#pragma unroll
          for (int e = 0; e < PART; ++e) g[e] = dy[u].get(h + e);
          if (a.kept) {
            from_kept16<PART>(z0[u].w + h / 2, f0);
            if (GATED) from_kept16<PART>(z1[u].w + h / 2, f1);
          } else {
#pragma unroll
            for (int e = 0; e < PART; ++e) {
              f0[e] = z0[u].get(h + e);
              if (GATED) f1[e] = z1[u].get(h + e);
            }
          }
          switch (a.act) {
            case CCE_ACT_RELU: grad_as<CCE_ACT_RELU, GATED>(d0, d1, g, f0, f1); break;
            case CCE_ACT_GELU: grad_as<CCE_ACT_GELU, GATED>(d0, d1, g, f0, f1); break;
            case CCE_ACT_GELU_TANH: grad_as<CCE_ACT_GELU_TANH, GATED>(d0, d1, g, f0, f1); break;
            case CCE_ACT_SILU: grad_as<CCE_ACT_SILU, GATED>(d0, d1, g, f0, f1); break;
            default: grad_as<CCE_ACT_NONE, GATED>(d0, d1, g, f0, f1); break;
          }
          set_part<T>(o0.w + h / 2, d0);
          if (GATED) set_part<T>(o1.w + h / 2, d1);
#pragma unroll
          for (int e = 0; e < PART; ++e) sum[h + e] += GATED ? 0.0f : d0[e];
        }
        if (a.dz[0]) o0.store(static_cast<T*>(a.dz[0]) + r * a.dz_pitch + col);
        if (GATED) o1.store(static_cast<T*>(a.dz[1]) + r * a.dz_pitch + col);
      }
    }
  }
  if constexpr (!GATED) {
    if (!a.part) return;
    __shared__ float sums[GROUPS][COLS * VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) sums[ty][tx * VEC + e] = sum[e];
    __syncthreads();
    for (int c = static_cast<int>(threadIdx.x); c < COLS * VEC; c += THREADS) {
      const int at = static_cast<int>(blockIdx.x) * COLS * VEC + c;
      if (at >= a.N) break;
      float t = 0.0f;
#pragma unroll
      for (int v = 0; v < GROUPS; ++v) t += sums[v][c];
      a.part[static_cast<int64_t>(blockIdx.y) * a.N + at] = t;
    }
  }
}

// Without products, beside which it is made otherwise.
__global__ void __launch_bounds__(32) sum_kernel(const __grid_constant__ LinSum a) {
  let_next_start();
  wait_for_previous();
  sum_columns(a, static_cast<int>(blockIdx.x) * 32 + static_cast<int>(threadIdx.x));
}

// --------------------------------------------------------------------- copies
// A warp's row.  The vectors of a row off 16 bytes are joined from two.
template <typename T>
__device__ __forceinline__ void copy_row(const cce_row_copy& c, int64_t row) {
  constexpr int VEC = 16 / sizeof(T);
  const int64_t outer = row / c.inner;
  const T* from = static_cast<const T*>(c.src) + outer * c.outer_stride + (row - outer * c.inner) * c.row_stride;
  T* to = static_cast<T*>(c.dst) + row * c.pitch;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(from) / sizeof(T)) & (VEC - 1);
  from -= shift;
#pragma unroll 4
  for (int64_t i = static_cast<int64_t>(threadIdx.x & 31) * VEC; i < c.cols; i += 32 * VEC) {
    Vec<T, VEC> lo, hi, v;
    lo.load(from + i);
    if (shift == 0) {
      v = lo;
    } else {
      hi.zero();
      if (i + VEC - shift < c.cols) hi.load(from + i + VEC);
      v.join(lo, hi, shift);
    }
    if (c.cols - i < VEC) v.keep(0, static_cast<int>(c.cols - i));
    v.store(to + i);
  }
}

__global__ void __launch_bounds__(THREADS) copy_kernel(const __grid_constant__ LinCopies a) {
  let_next_start();
  wait_for_previous();
  const int64_t step = static_cast<int64_t>(gridDim.x) * (THREADS / 32);
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * (THREADS / 32) + (threadIdx.x >> 5); r < a.rows; r += step) {
    int m = 0;
    while (m + 1 < a.n && r >= a.first[m + 1]) ++m;
    if (a.c[m].bytes == 4) {
      copy_row<float>(a.c[m], r - a.first[m]);
    } else {
      copy_row<__nv_bfloat16>(a.c[m], r - a.first[m]);
    }
  }
}

bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }

// Blocks for the rows: six an SM in all, no more than there are rows for.
int grad_rows(int64_t M, int64_t N, int vec) {
  const int64_t x = (N + COLS * vec - 1) / (COLS * vec);
  return static_cast<int>(std::max<int64_t>(
      1, std::min({int64_t(LIN_GRAD_PARTS), (6 * LIN_SMS + x - 1) / x, (M + GROUPS * UNROLL - 1) / (GROUPS * UNROLL)})));
}

template <typename T, typename TY, bool GATED>
cudaError_t launch_grad(const LinGrad& a, cudaStream_t s, int* parts) {
  // vectors of 8: whole rows of them at 16 bytes in every matrix (dy of fp32 rows as two)
  bool wide = a.N % 8 == 0 && a.dy_pitch % 8 == 0 && multiple(a.dy, 16);
  for (int m = 0; m < (GATED ? 2 : 1); ++m) {
    if (a.z[m]) wide = wide && a.z_pitch[m] % 8 == 0 && multiple(a.z[m], 16);
    if (a.dz[m]) wide = wide && a.dz_pitch % 8 == 0 && multiple(a.dz[m], 16);
  }
  const int vec = wide ? 8 : 1;
  const int x = (a.N + COLS * vec - 1) / (COLS * vec), y = grad_rows(a.M, a.N, vec);
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
  *parts = y;
  return wide ? launch_after(grad_kernel<T, TY, GATED, 8>, grid, dim3(THREADS), 0, 1, s, a)
              : launch_after(grad_kernel<T, TY, GATED, 1>, grid, dim3(THREADS), 0, 1, s, a);
}

template <typename T>
cudaError_t launch_grad_of(const LinGrad& a, bool gated, cudaStream_t s, int* parts) {
  if (gated) return launch_grad<T, T, true>(a, s, parts);
  return a.dy_type == CCE_F32 ? launch_grad<T, float, false>(a, s, parts) : launch_grad<T, T, false>(a, s, parts);
}

template <typename T, bool GATED>
cudaError_t launch_join(const LinProblem& p, int sms, cudaStream_t s) {
  const LinEpilogue& e = p.e;
  const auto fits = [](const void* m, int64_t pitch, int64_t bytes) { return !m || (pitch % 4 == 0 && multiple(m, 4 * bytes)); };
  const int64_t y_bytes = e.y_type == CCE_F32 ? 4 : 2;
  const bool wide = p.I % 4 == 0 && fits(e.y, e.y_pitch, y_bytes) && fits(e.res, e.res_pitch | e.res_outer, y_bytes) &&
                    fits(e.z[0], e.z_pitch, 2) && fits(e.z[1], e.z_pitch, 2) &&
                    fits(e.bias, 0, e.bias_type == CCE_F32 ? 4 : 2);
  const int cols = JOIN_COLS * (wide ? 4 : 1), rows = THREADS / JOIN_COLS;
  const int x = (p.I + cols - 1) / cols;
  const int y = std::max(1, std::min((p.J + rows - 1) / rows, (16 * sms + x - 1) / x));
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y));
  const float* part = p.part;
  return wide ? launch_after(join_kernel<T, GATED, 4>, grid, dim3(THREADS), 0, 1, s, part, p.I, p.J, p.splits, e)
              : launch_after(join_kernel<T, GATED, 1>, grid, dim3(THREADS), 0, 1, s, part, p.I, p.J, p.splits, e);
}

}  // namespace

cudaError_t launch_linear_join(const LinProblem& p, bool gated, bool bf16, int sms, cudaStream_t s) {
  if (bf16) return gated ? launch_join<__nv_bfloat16, true>(p, sms, s) : launch_join<__nv_bfloat16, false>(p, sms, s);
  return gated ? launch_join<__half, true>(p, sms, s) : launch_join<__half, false>(p, sms, s);
}

int linear_grad_parts(int64_t M, int64_t N) { return grad_rows(M, N, 8); }

cudaError_t launch_linear_grad(const LinGrad& a, bool gated, bool bf16, cudaStream_t s, int* parts) {
  return bf16 ? launch_grad_of<__nv_bfloat16>(a, gated, s, parts) : launch_grad_of<__half>(a, gated, s, parts);
}

cudaError_t launch_linear_copies(const LinCopies& a, int sms, cudaStream_t s) {
  const int64_t blocks = (a.rows + THREADS / 32 - 1) / (THREADS / 32);
  return launch_after(copy_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 8 * sms))), dim3(THREADS), 0, 1, s, a);
}

cudaError_t launch_linear_sum(const LinSum& a, cudaStream_t s) {
  return launch_after(sum_kernel, dim3(static_cast<unsigned>((a.N + 31) / 32)), dim3(32), 0, 1, s, a);
}

}  // namespace cce

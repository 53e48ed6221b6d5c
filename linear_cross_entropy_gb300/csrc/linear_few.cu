// A layer over few rows (decoding): out[j][i] = epilogue(sum over k of w[i][k] x[j][k])
// for up to 32 rows j.
//
// Bound by reading the weights once, so nothing is staged: a warp reads 16-byte
// vectors of 16 weight rows straight into the fragments of mma.m16n8k16, whose k
// index is free to be permuted as long as both operands are permuted alike.  (A
// tcgen05 MMA wants its operands in shared memory and 128 weight rows a CTA, and
// there are too few of those to keep 152 SMs reading.)  The eight warps of a block
// take every eighth 64 of k and add up through shared memory in a fixed order.
// One row of 896 x 896 takes 2.5 us, a launch's own time; 13 rows of 4,096 x 4,096
// 6.7 us, 5.0 TB/s.
#include "internal.h"
#include "linear.h"
#include "linear_epilogue.cuh"

#include <type_traits>

namespace cce {
namespace {

constexpr int WARPS = 8;
constexpr int ROWS = 16;  // of w, a block

template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}

// Eight values from k on, zeros behind K: what lies there may be anything.
__device__ __forceinline__ uint4 vector_at(const uint16_t* row, int k, int K) {
  if (k >= K) return make_uint4(0u, 0u, 0u, 0u);
  uint4 v = *reinterpret_cast<const uint4*>(row + k);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
  const int n = K - k;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < n ? w[i] : 2 * i < n ? w[i] & 0xffffu : 0u;
  return v;
}

// 32 of k of the fragments: thread t of a row has 8t .. 8t + 7, of which the first four are one MMA's, the others the
// next one's.
template <bool BF16, int NT, int MATS>
struct Step {
  uint4 w[MATS][2], x[NT];

  // INSIDE: all of them are below K, and the loads of several steps are in flight at once.
  template <bool INSIDE>
  __device__ __forceinline__ void load(const uint16_t* const (&wp)[MATS][2], const uint16_t* const (&xp)[NT], int k, int K) {
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[m][h] = INSIDE ? *reinterpret_cast<const uint4*>(wp[m][h] + k) : vector_at(wp[m][h], k, K);
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = INSIDE ? *reinterpret_cast<const uint4*>(xp[n] + k) : vector_at(xp[n], k, K);
  }
  __device__ __forceinline__ void add_to(float (&c)[MATS][NT][4]) const {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        mma<BF16>(c[m][n], w[m][0].x, w[m][1].x, w[m][0].y, w[m][1].y, x[n].x, x[n].y);
        mma<BF16>(c[m][n], w[m][0].z, w[m][1].z, w[m][0].w, w[m][1].w, x[n].z, x[n].w);
      }
    }
  }
};

// PARTS: fp32 results of a long K.  mma.sync cuts where it could round, as tcgen05.mma does: a warp's sum goes on in other
// registers every LIN_CHUNK_K of its k, and the parts are added to nearest, where they wait in shared memory.  With K = 65,536
// a sum is 1.0e-6 of the norm off and not 9.1e-6.  (In kernels of their own: in all it cost a gated layer of 32 rows 7%.)
template <bool BF16, int NT, bool GATED, bool PARTS>
__global__ void __launch_bounds__(32 * WARPS, 2) few_kernel(const __grid_constant__ LinFew a) {
  constexpr int MATS = GATED ? 2 : 1;
  constexpr int UNROLL = GATED ? 2 : 4;  // steps in flight: eight vectors of the weights a thread
  __shared__ float sums[WARPS][MATS][ROWS][8 * NT + 1];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, t = lane & 3;
  const int i0 = static_cast<int>(blockIdx.x) * ROWS;
  let_next_start();
  wait_for_previous();
  // rows behind the last one, of w and of x, are read as the last one, and their results not written
  const uint16_t* w[MATS][2];
#pragma unroll
  for (int m = 0; m < MATS; ++m) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[m][h] = static_cast<const uint16_t*>(a.w[m]) + static_cast<int64_t>(min(i0 + g + 8 * h, a.I - 1)) * a.w_pitch[m];
  }
  const uint16_t* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    x[n] = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(min(g + 8 * n, a.J - 1)) * a.x_pitch;

  float c[MATS][NT][4] = {};
  bool first = true;
  const auto put_aside = [&] {
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float& to = sums[warp][m][g + 8 * (q >> 1)][8 * n + 2 * t + (q & 1)];
          to = PARTS && !first ? to + c[m][n][q] : c[m][n][q];
          if (PARTS) c[m][n][q] = 0.0f;
        }
    first = false;
  };
  int left = LIN_CHUNK_K / 64;
  // a warp's k: two steps at 64 (warp + WARPS q), q = 0, 1, ...
  constexpr int STRIDE = 64 * WARPS;
  int k = warp * 64 + 8 * t;
  const int last = a.K - 64 + 8 * t;  // the last k whose two steps are inside
#pragma unroll 1
  for (; k + STRIDE * (UNROLL / 2 - 1) <= last; k += STRIDE * (UNROLL / 2)) {
    Step<BF16, NT, MATS> s[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) s[u].template load<true>(w, x, k + (u >> 1) * STRIDE + (u & 1) * 32, a.K);
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) s[u].add_to(c);
    if (PARTS && (left -= UNROLL / 2) == 0) {
      put_aside();
      left = LIN_CHUNK_K / 64;
    }
  }
#pragma unroll 1
  for (; k - 8 * t < a.K; k += STRIDE) {
    Step<BF16, NT, MATS> s[2];
    if (k <= last) {
      s[0].template load<true>(w, x, k, a.K);
      s[1].template load<true>(w, x, k + 32, a.K);
    } else {
      s[0].template load<false>(w, x, k, a.K);
      s[1].template load<false>(w, x, k + 32, a.K);
    }
    s[0].add_to(c);
    s[1].add_to(c);
  }
  put_aside();
  __syncthreads();
  const int r = static_cast<int>(threadIdx.x) % ROWS, i = i0 + r;
  if (i >= a.I) return;
  for (int j = static_cast<int>(threadIdx.x) / ROWS; j < min(8 * NT, a.J); j += 32 * WARPS / ROWS) {
    float z0[1] = {0.0f}, z1[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < WARPS; ++v) {
      z0[0] += sums[v][0][r][j];
      if (GATED) z1[0] += sums[v][MATS - 1][r][j];
    }
    finish_row<typename std::conditional<BF16, __nv_bfloat16, __half>::type, GATED>(a.e, j, i, z0, z1);
  }
}

template <bool BF16, int NT>
cudaError_t launch(const LinFew& a, bool gated, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.I + ROWS - 1) / ROWS)), block(32 * WARPS);
  if (gated) return launch_after(few_kernel<BF16, NT, true, false>, grid, block, 0, 1, s, a);
  return a.e.y_type == CCE_F32 && a.K > WARPS * LIN_CHUNK_K ? launch_after(few_kernel<BF16, NT, false, true>, grid, block, 0, 1, s, a)
                                                            : launch_after(few_kernel<BF16, NT, false, false>, grid, block, 0, 1, s, a);
}

}  // namespace

cudaError_t launch_linear_few(const LinFew& a, bool gated, bool bf16, cudaStream_t s) {
  const int tiles = (a.J + 7) / 8;
  if (bf16)
    return tiles == 1   ? launch<true, 1>(a, gated, s)
           : tiles == 2 ? launch<true, 2>(a, gated, s)
                        : launch<true, 4>(a, gated, s);
  return tiles == 1   ? launch<false, 1>(a, gated, s)
         : tiles == 2 ? launch<false, 2>(a, gated, s)
                      : launch<false, 4>(a, gated, s);
}

}  // namespace cce

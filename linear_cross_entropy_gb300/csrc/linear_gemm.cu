// Persistent, warp-specialised tcgen05 GEMM of the layers in front of the head:
//
//   out[j][i] = epilogue(sum over k of A(i, k) B(j, k))
//
// A holds what becomes the contiguous index of the output (weights in the
// forward pass, so that a thread of the epilogue has one output column, its bias
// in a register, and a warp writes 32 neighbouring values of a row: no staging in
// shared memory and no alignment of the output), B its rows (tokens).  Either may
// be stored with k contiguous or with its own index contiguous:
//
//   forward          A = W  [N, K] along k       B = x  [M, K] along k
//   dx = dz W        A = W  [N, K] along i = K   B = dz [M, N] along k = N
//   dW = dz^T x      A = x  [M, K] along i = K   B = dz [M, N] along j = N
//
// Up to three products run in one launch (dx and both dW of a gated layer).  A
// gated forward has two accumulators a tile, gate and up, whose A tiles share
// the B tile; dx of a gated layer runs one sum over two pairs of operands.
//
// Roles (320 threads): warp 0 lane 0 loads (TMA, 64-deep stages, as many as fit in
// 192 KiB), warp 1 lane 0 issues tcgen05.mma into one of two TMEM accumulators, warps 2
// to 9 are the epilogue (warp w reads TMEM lanes 32 (w % 4) to + 31, and every
// second 32 columns).  CTA pairs share an MMA of M = 256: each CTA holds 128 rows
// of A and half of B's columns.
//
// Bound by the tensor cores for many rows, and by reading the weights for few.
#include "gemm_args.h"
#include "internal.h"
#include "linear.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace cce {
namespace {

constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int ACC_COLS = 256;  // TMEM columns of one of the two accumulators
constexpr int RING_BYTES = 192 * 1024;
constexpr int MAX_RING = 12;
constexpr int A_BYTES = LIN_BI * LIN_BK * 2;  // one A tile of a stage
constexpr int SMEM = 1024 + RING_BYTES + 512;

__device__ int32_t linear_error;  // CCE_DEVERR_* of waits that ran out

struct Shared {
  uint8_t* ring;
  uint64_t* full;       // [MAX_RING]
  uint64_t* empty;      // [MAX_RING]
  uint64_t* acc_full;   // [2]
  uint64_t* acc_empty;  // [2]
  uint64_t* drain;
  uint32_t* tmem;
  int* abort_flag;
};

__device__ __forceinline__ Shared carve(uint8_t* raw) {
  Shared s;
  s.ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.full = reinterpret_cast<uint64_t*>(s.ring + RING_BYTES);
  s.empty = s.full + MAX_RING;
  s.acc_full = s.empty + MAX_RING;
  s.acc_empty = s.acc_full + 2;
  s.drain = s.acc_empty + 2;
  s.tmem = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort_flag = reinterpret_cast<int*>(s.tmem + 1);
  return s;
}
static_assert(8 * (2 * MAX_RING + 5) + 8 <= 512, "barriers fit");

struct Tile {
  const LinProblem* p;
  int it, jt, split;
  int kb, kb_end;  // blocks of K
};

__device__ __forceinline__ Tile tile_of(const LinArgs& a, int item) {
  int q = 0;
  while (q + 1 < a.problems && item >= a.p[q].items) item -= a.p[q++].items;
  Tile t;
  t.p = &a.p[q];
  const LinProblem& p = *t.p;
  // groups of i tiles, inside of which i runs fastest, then j, then the splits: tiles that
  // run at the same time share rows of A and of B in L2
  const int per_split = p.i_tiles * p.j_tiles;
  t.split = item / per_split;
  item -= t.split * per_split;
  const int per_group = p.group * p.j_tiles;
  const int g = item / per_group;
  item -= g * per_group;
  const int width = min(p.group, p.i_tiles - g * p.group);
  t.jt = item / width;
  t.it = g * p.group + item - t.jt * width;
  t.kb = t.split * p.kb_split;
  t.kb_end = min(p.kb_all, t.kb + p.kb_split);
  return t;
}

// Bytes of a CTA's B tile in a stage, and of a stage.
template <bool PAIR>
__device__ __forceinline__ int b_rows(const LinProblem& p) {
  return PAIR ? p.jt / 2 : p.jt;
}

template <bool PAIR, bool GATED>
struct Ring {
  // of the widest tile
  static constexpr int kBytes = (GATED ? 2 : 1) * A_BYTES + (GATED ? 128 : 256) / (PAIR ? 2 : 1) * LIN_BK * 2;
  static constexpr int kStages = RING_BYTES / kBytes < MAX_RING ? RING_BYTES / kBytes : MAX_RING;
};

template <bool PAIR>
__device__ __forceinline__ void load_box(const CUtensorMap* m, uint64_t* bar, uint32_t lead, uint8_t* to, int x, int y) {
  if constexpr (PAIR) {
    tma_load_2d_pair(m, lead, to, x, y);
  } else {
    tma_load_2d(m, bar, to, x, y);
  }
}

template <bool PAIR, bool GATED>
__device__ __forceinline__ void load_loop(const LinArgs& a, const Shared& s) {
  using R = Ring<PAIR, GATED>;
  volatile int* abort_flag = s.abort_flag;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const uint32_t lead = PAIR ? mapa_shared(smem_u32(s.full), 0) : 0u;
  int stage = 0;
  uint32_t phase = 0;
  uint32_t issued = 0, issued_par = 0;  // per stage: ever issued, parity of its last phase
  bool ok = true;
  for (int item = unit; ok && item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const int rows = b_rows<PAIR>(p);
    const int i0 = t.it * (PAIR ? 2 * LIN_BI : LIN_BI) + rank * LIN_BI;
    const int j0 = t.jt * p.jt + rank * rows;
    const uint32_t bytes = static_cast<uint32_t>(((GATED ? 2 : 1) * A_BYTES + rows * LIN_BK * 2) * (PAIR ? 2 : 1));
    for (int kb = t.kb; kb < t.kb_end; ++kb) {
      if (!wait_bounded(&s.empty[stage], phase ^ 1u, abort_flag, &linear_error)) {
        ok = false;
        break;
      }
      uint64_t* bar = &s.full[stage];
      const uint32_t bar_lead = lead + 8u * static_cast<uint32_t>(stage);
      uint8_t* to = s.ring + stage * R::kBytes;
      const int part = kb >= p.kb_first ? 1 : 0;
      const int k0 = (part ? kb - p.kb_first : kb) * LIN_BK;
      if (rank == 0) mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
      for (int g = 0; g < (GATED ? 2 : 1); ++g) {
        const CUtensorMap* m = &p.a[GATED ? g : part];
        if (p.a_mn) {  // two groups of 64 i, one row of 128 bytes for each k
          load_box<PAIR>(m, bar, bar_lead, to, i0, k0);
          load_box<PAIR>(m, bar, bar_lead, to + A_BYTES / 2, i0 + 64, k0);
        } else {
          load_box<PAIR>(m, bar, bar_lead, to, k0, i0);
        }
        to += A_BYTES;
      }
      const CUtensorMap* m = &p.b[part];
      if (p.b_mn) {
        for (int r = 0; r < rows; r += 64) load_box<PAIR>(m, bar, bar_lead, to + r * LIN_BK * 2, j0 + r, k0);
      } else {
        load_box<PAIR>(m, bar, bar_lead, to, k0, j0);
      }
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == R::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  }
  if (!*abort_flag) return;
  if (PAIR && rank != 0) {
    // this CTA's copies complete on the other's barriers: 10 ms for those in flight
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 10000000ull) {
    }
  } else {
    for (int i = 0; i < R::kStages; ++i) {
      if (issued & (1u << i)) {
        volatile int none = 0;
        wait_bounded(&s.full[i], (issued_par >> i) & 1u, &none, nullptr);
      }
    }
  }
}

template <bool PAIR, bool GATED>
__device__ __forceinline__ void mma_loop(const LinArgs& a, const Shared& s, uint32_t tmem) {
  if (PAIR && cluster_ctarank() != 0) return;  // the even CTA issues for both
  using R = Ring<PAIR, GATED>;
  volatile int* abort_flag = s.abort_flag;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool any = false, ok = true;
  for (int item = unit; ok && item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const bool a_mn = p.a_mn, b_mn = p.b_mn;
    // bits 7-9 and 10-12 of the descriptor: 1 = bf16, 0 = fp16
    const uint32_t idesc = idesc_bf16(PAIR ? 2 * LIN_BI : LIN_BI, p.jt, a_mn, b_mn) & (a.bf16 ? ~0u : ~((1u << 7) | (1u << 10)));
    // along its own index: 64-element groups of 64 rows of 128 bytes, 16 of k are 16 rows; along
    // k: 16 of k are 32 bytes of a row
    const uint32_t a_lbo = a_mn ? LIN_BK * 128u : 16u, b_lbo = b_mn ? LIN_BK * 128u : 16u;
    const uint64_t a_step = a_mn ? 2048u >> 4 : 32u >> 4, b_step = b_mn ? 2048u >> 4 : 32u >> 4;
    if (!wait_bounded(&s.acc_empty[acc], acc_phase ^ 1u, abort_flag, &linear_error)) break;
    tc_fence_after();
    const uint32_t d = tmem + static_cast<uint32_t>(acc * ACC_COLS);
    uint32_t accumulate = 0;
    for (int kb = t.kb; kb < t.kb_end; ++kb) {
      if (!wait_bounded(&s.full[stage], phase, abort_flag, &linear_error)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int part = kb >= p.kb_first ? 1 : 0;
      const int left = p.klen[part] - (part ? kb - p.kb_first : kb) * LIN_BK;
      const int steps = left >= LIN_BK ? LIN_BK / 16 : (left + 15) / 16;  // behind K's end there are zeros
      const uint32_t at = smem_u32(s.ring + stage * R::kBytes);
      const uint64_t b_desc = smem_desc_sw128(at + (GATED ? 2 : 1) * A_BYTES, b_lbo, 1024u);
#pragma unroll
      for (int g = 0; g < (GATED ? 2 : 1); ++g) {
        const uint64_t a_desc = smem_desc_sw128(at + g * A_BYTES, a_lbo, 1024u);
        const uint32_t to = d + static_cast<uint32_t>(g * ACC_COLS / 2);
#pragma unroll
        for (int k = 0; k < LIN_BK / 16; ++k) {
          if (k < steps) {
            if constexpr (PAIR) {
              mma_bf16_pair(to, a_desc + a_step * k, b_desc + b_step * k, idesc, accumulate | (k > 0));
            } else {
              mma_bf16(to, a_desc + a_step * k, b_desc + b_step * k, idesc, accumulate | (k > 0));
            }
          }
        }
      }
      accumulate = 1;
      any = true;
      if constexpr (PAIR) {
        mma_commit_pair_both(&s.empty[stage]);
      } else {
        mma_commit(&s.empty[stage]);
      }
      if (++stage == R::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (!ok) break;
    if constexpr (PAIR) {
      mma_commit_pair_both(&s.acc_full[acc]);
    } else {
      mma_commit(&s.acc_full[acc]);
    }
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (*abort_flag && any) {
    if constexpr (PAIR) {
      mma_commit_pair_local(s.drain);
    } else {
      mma_commit(s.drain);
    }
    volatile int none = 0;
    wait_bounded(s.drain, 0, &none, nullptr);
  }
}

template <bool PAIR, bool GATED>
__device__ __forceinline__ void epilogue_loop(const LinArgs& a, const Shared& s, uint32_t tmem, int warp) {
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int quarter = warp & 3, half = (warp - 2) >> 2;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t release = PAIR ? mapa_shared(smem_u32(s.acc_empty), 0) : smem_u32(s.acc_empty);
  int acc = 0;
  uint32_t acc_phase = 0;
  for (int item = unit; item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const int i = t.it * (PAIR ? 2 * LIN_BI : LIN_BI) + rank * LIN_BI + quarter * 32 + static_cast<int>(lane_id());
    const bool inside = i < p.I;
    const float bias = p.e.bias && p.splits == 1 && inside ? load_scalar(p.e.bias, p.e.bias_type, i) : 0.0f;
    if (!warp_wait_bounded(&s.acc_full[acc], acc_phase, s.abort_flag, &linear_error)) break;
    tc_fence_after();
    const uint32_t from = lane_base + static_cast<uint32_t>(acc * ACC_COLS);
    for (int c = half; c < p.jt / 32; c += 2) {
      const int j0 = t.jt * p.jt + 32 * c;
      const int n = min(32, p.J - j0);
      if (n <= 0) break;  // the same in all lanes
      uint32_t r0[32], r1[32];
      __syncwarp();  // the lanes outside of the matrix are back
      tmem_ld32(from + 32 * c, r0);
      if constexpr (GATED) tmem_ld32(from + ACC_COLS / 2 + 32 * c, r1);
      tmem_ld_wait();
      if (!inside) continue;
      if (p.splits > 1) {  // a partial sum
        float* to = p.part + (static_cast<int64_t>(t.split * (GATED ? 2 : 1)) * p.J + j0) * p.I + i;
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          if (u < n) {
            to[static_cast<int64_t>(u) * p.I] = __uint_as_float(r0[u]);
            if constexpr (GATED) to[(static_cast<int64_t>(p.J) + u) * p.I] = __uint_as_float(r1[u]);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {  // in two halves: a whole column with its residual spills
          float z0[16], z1[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            z0[u] = __uint_as_float(r0[h + u]);
            if constexpr (GATED) z1[u] = __uint_as_float(r1[h + u]);
          }
          if (h < n) finish_column<GATED>(p.e, a.bf16, bias, i, j0 + h, n - h, z0, z1);
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane_id() == 0) {
      if constexpr (PAIR) {
        mbar_arrive_cluster(release + 8u * static_cast<uint32_t>(acc));
      } else {
        mbar_arrive(&s.acc_empty[acc]);
      }
    }
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
}

template <bool PAIR, bool GATED>
__global__ void __launch_bounds__(THREADS, 1) linear_kernel(const __grid_constant__ LinArgs a) {
  extern __shared__ uint8_t raw[];
  const Shared s = carve(raw);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  let_next_start();
  if (threadIdx.x == 0) {
    for (int i = 0; i < Ring<PAIR, GATED>::kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], PAIR ? 2 * EPI_WARPS : EPI_WARPS);
    }
    mbar_init(s.drain, 1);
    *s.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(s.tmem, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(s.tmem, TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // the other CTA's barriers exist before anything reaches them
  tc_fence_after();
  const uint32_t tmem = *s.tmem;
  wait_for_previous();

  if (warp == 0) {
    if (lane_id() == 0) load_loop<PAIR, GATED>(a, s);
  } else if (warp == 1) {
    if (lane_id() == 0) mma_loop<PAIR, GATED>(a, s, tmem);
  } else {
    epilogue_loop<PAIR, GATED>(a, s, tmem, warp);
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync();  // no CTA leaves while the other may still signal its barriers
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) {
      tmem_dealloc_pair(tmem, TMEM_COLS);
    } else {
      tmem_dealloc(tmem, TMEM_COLS);
    }
  }
}

template <bool PAIR, bool GATED>
cudaError_t set_shared() {
  return cudaFuncSetAttribute(linear_kernel<PAIR, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
}

}  // namespace

cudaError_t prepare_linear_gemm() {
  cudaError_t e = set_shared<false, false>();
  if (e == cudaSuccess) e = set_shared<false, true>();
  if (e == cudaSuccess) e = set_shared<true, false>();
  if (e == cudaSuccess) e = set_shared<true, true>();
  return e;
}

int linear_pair_units(int sms) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, linear_kernel<true, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_linear_gemm(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(pair ? 2 * units : units)), block(THREADS);
  const unsigned cluster = pair ? 2 : 1;
  if (pair) {
    return gated ? launch_after(linear_kernel<true, true>, grid, block, SMEM, cluster, s, a)
                 : launch_after(linear_kernel<true, false>, grid, block, SMEM, cluster, s, a);
  }
  return gated ? launch_after(linear_kernel<false, true>, grid, block, SMEM, cluster, s, a)
               : launch_after(linear_kernel<false, false>, grid, block, SMEM, cluster, s, a);
}

cudaError_t take_linear_error(int32_t* word, cudaStream_t s) {
  const int32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(word, linear_error, sizeof zero, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && *word != 0) {
    e = cudaMemcpyToSymbolAsync(linear_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e;
}

}  // namespace cce

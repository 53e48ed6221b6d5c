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
// Up to three products run in one launch (dx and both dW of a gated layer); dx of a
// gated layer is one sum over two pairs of operands.  A gated forward's 128 MMA
// rows are 64 of each weight, so that its loads and MMAs are those of a layer twice
// as wide; the warps that hold a gate's rows and those with the up projection's
// exchange half of their values in shared memory.
//
// Roles (576 threads): warp 0 lane 0 loads (TMA; a pair's stages are 128 deep in K, a
// single CTA's 64, as many as fit in 192 KiB), warp 1 lane 0 issues tcgen05.mma into
// one of two TMEM accumulators, the other 16 warps are the epilogue (warp w reads TMEM
// lanes 32 (w % 4) to + 31, and every fourth 16 columns).  CTA pairs share an MMA of
// M = 256: each CTA holds 128 rows of A and half of B's columns.
//
// Bound by the tensor cores for many rows, and by reading the weights for few.
#include "gemm_args.h"
#include "internal.h"
#include "linear.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace cce {
namespace {

constexpr int EPI_WARPS = 16;
constexpr int PHASES = EPI_WARPS / 4;  // warps that share the columns of 32 TMEM lanes
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int ACC_COLS = 256;  // TMEM columns of one of the two accumulators
constexpr int CHUNK = 16;      // columns that a warp reads at a time
constexpr int HALF = CHUNK / 2;
constexpr int GROUP = 64 * 128;  // bytes of 64 rows of 128 bytes
// gated: what a warp hands over, twice
constexpr int SWAP_BYTES = 2 * HALF * 32 * 4;
constexpr int BAR_BYTES_LIN = 512;

template <bool GATED>
constexpr int shared_bytes() {
  return 1024 + LIN_RING_BYTES + BAR_BYTES_LIN + (GATED ? EPI_WARPS * SWAP_BYTES : 0);
}
static_assert(shared_bytes<true>() <= 227 * 1024, "shared memory of a CTA");

__device__ int32_t linear_error;  // CCE_DEVERR_* of waits that ran out

struct Shared {
  uint8_t* ring;
  uint64_t* full;       // [LIN_MAX_STAGES]
  uint64_t* empty;      // [LIN_MAX_STAGES]
  uint64_t* acc_full;   // [2]
  uint64_t* acc_empty;  // [2]
  uint64_t* drain;
  uint32_t* tmem;
  int* abort_flag;
  float* swap;  // gated: [EPI_WARPS][2][HALF][32]
};

__device__ __forceinline__ Shared carve(uint8_t* raw) {
  Shared s;
  s.ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.full = reinterpret_cast<uint64_t*>(s.ring + LIN_RING_BYTES);
  s.empty = s.full + LIN_MAX_STAGES;
  s.acc_full = s.empty + LIN_MAX_STAGES;
  s.acc_empty = s.acc_full + 2;
  s.drain = s.acc_empty + 2;
  s.tmem = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort_flag = reinterpret_cast<int*>(s.tmem + 1);
  s.swap = reinterpret_cast<float*>(s.ring + LIN_RING_BYTES + BAR_BYTES_LIN);
  return s;
}
static_assert(8 * (2 * LIN_MAX_STAGES + 5) + 8 <= BAR_BYTES_LIN, "barriers fit");

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

// A box to `to`, whose bytes are counted on the stage's barrier (of a pair: the even CTA's).
template <bool PAIR>
struct Loader {
  uint64_t* bar;
  uint32_t lead;  // the barrier's cluster address

  __device__ __forceinline__ void box2(const CUtensorMap* m, uint8_t* to, int x, int y) const {
    if constexpr (PAIR) {
      tma_load_2d_pair(m, lead, to, x, y);
    } else {
      tma_load_2d(m, bar, to, x, y);
    }
  }
  __device__ __forceinline__ void box3(const CUtensorMap* m, uint8_t* to, int x, int y, int z) const {
    if constexpr (PAIR) {
      tma_load_3d_pair(m, lead, to, x, y, z);
    } else {
      tma_load_3d(m, bar, to, x, y, z);
    }
  }
  // `rows` rows from r0 on of an operand, the block of K at k0.  Along k: 64 of k are
  // `pitch` bytes apart; along its own index: 64 of them.
  __device__ __forceinline__ void operand(const CUtensorMap* m, bool mn, bool whole, uint8_t* to, int r0, int rows,
                                          int k0, int pitch) const {
    constexpr int BK = lin_bk(PAIR);
    if (mn) {
      if (whole) {
        box3(m, to, 0, k0, r0 >> 6);
      } else {
        for (int r = 0; r < rows; r += 64) box2(m, to + r * 2 * BK, r0 + r, k0);
      }
    } else if (whole) {
      box3(m, to, 0, r0, k0 >> 6);
    } else {
#pragma unroll
      for (int k = 0; k < BK; k += 64) box2(m, to + (k >> 6) * pitch, k0 + k, r0);
    }
  }
};

template <bool PAIR, bool GATED>
__device__ __forceinline__ void load_loop(const LinArgs& a, const Shared& s) {
  constexpr int BK = lin_bk(PAIR), A_BYTES = LIN_BI * BK * 2;
  volatile int* abort_flag = s.abort_flag;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const uint32_t lead = PAIR ? mapa_shared(smem_u32(s.full), 0) : 0u;
  const int stages = a.stages, stage_bytes = a.stage_bytes;
  int stage = 0;
  uint32_t phase = 0;
  uint32_t issued = 0, issued_par = 0;  // per stage: ever issued, parity of its last phase
  bool ok = true;
  for (int item = unit; ok && item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const bool a_mn = p.a_mn, b_mn = p.b_mn, a_3d = p.a_3d, b_3d = p.b_3d;
    const int rows = PAIR ? p.jt / 2 : p.jt;
    const int i0 = (t.it * (PAIR ? 2 : 1) + rank) * (GATED ? LIN_BI / 2 : LIN_BI);
    const int j0 = t.jt * p.jt + rank * rows;
    const uint32_t bytes = static_cast<uint32_t>((A_BYTES + rows * BK * 2) * (PAIR ? 2 : 1));
    for (int kb = t.kb; kb < t.kb_end; ++kb) {
      if (!wait_bounded_long(&s.empty[stage], phase ^ 1u, abort_flag, &linear_error)) {
        ok = false;
        break;
      }
      const Loader<PAIR> load{&s.full[stage], lead + 8u * static_cast<uint32_t>(stage)};
      uint8_t* to = s.ring + stage * stage_bytes;
      if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], bytes);
      const int part = !GATED && kb >= p.kb_first ? 1 : 0;
      const int k0 = (part ? kb - p.kb_first : kb) * BK;
      if constexpr (GATED) {
        load.operand(&p.a[0], false, false, to, i0, 64, k0, 2 * GROUP);
        load.operand(&p.a[1], false, false, to + GROUP, i0, 64, k0, 2 * GROUP);
      } else {
        load.operand(&p.a[part], a_mn, a_3d, to, i0, LIN_BI, k0, 2 * GROUP);
      }
      load.operand(&p.b[part], b_mn, b_3d, to + A_BYTES, j0, rows, k0, rows * 128);
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == stages) {
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
    for (int i = 0; i < stages; ++i) {
      if (issued & (1u << i)) {
        volatile int none = 0;
        wait_bounded_long(&s.full[i], (issued_par >> i) & 1u, &none, nullptr);
      }
    }
  }
}

template <bool PAIR>
__device__ __forceinline__ void mma_loop(const LinArgs& a, const Shared& s, uint32_t tmem) {
  if (PAIR && cluster_ctarank() != 0) return;  // the even CTA issues for both
  constexpr int BK = lin_bk(PAIR), A_BYTES = LIN_BI * BK * 2;
  volatile int* abort_flag = s.abort_flag;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int stages = a.stages, stage_bytes = a.stage_bytes;
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool any = false, ok = true;
  for (int item = unit; ok && item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const bool a_mn = p.a_mn, b_mn = p.b_mn;
    // bits 7-9 and 10-12 of the descriptor: 1 = bf16, 0 = fp16
    const uint32_t idesc = idesc_bf16(PAIR ? 2 * LIN_BI : LIN_BI, p.jt, a_mn, b_mn) & (a.bf16 ? ~0u : ~((1u << 7) | (1u << 10)));
    // along its own index: 64-element groups of BK rows of 128 bytes, 16 of k are 16 rows; along
    // k: 16 of k are 32 bytes of a row, 64 of k all rows
    const uint32_t a_lbo = a_mn ? BK * 128u : 16u, b_lbo = b_mn ? BK * 128u : 16u;
    const uint32_t a_step = (a_mn ? 2048u : 32u) >> 4, b_step = (b_mn ? 2048u : 32u) >> 4;
    const uint32_t a_next = (a_mn ? 8192u : 2u * GROUP) >> 4;
    const uint32_t b_next = (b_mn ? 8192u : (PAIR ? p.jt / 2 : p.jt) * 128u) >> 4;
    if (!wait_bounded_long(&s.acc_empty[acc], acc_phase ^ 1u, abort_flag, &linear_error)) break;
    tc_fence_after();
    const uint32_t d = tmem + static_cast<uint32_t>(acc * ACC_COLS);
    uint32_t accumulate = 0;
    for (int kb = t.kb; kb < t.kb_end; ++kb) {
      if (!wait_bounded_long(&s.full[stage], phase, abort_flag, &linear_error)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int part = kb >= p.kb_first ? 1 : 0;
      const int left = p.klen[part] - (part ? kb - p.kb_first : kb) * BK;
      const uint32_t at = smem_u32(s.ring + stage * stage_bytes);
      const uint64_t a_desc = smem_desc_sw128(at, a_lbo, 1024u);
      const uint64_t b_desc = smem_desc_sw128(at + A_BYTES, b_lbo, 1024u);
      const auto mma = [&](int k) {
        const uint64_t ad = a_desc + (k >> 2) * a_next + (k & 3) * a_step, bd = b_desc + (k >> 2) * b_next + (k & 3) * b_step;
        if constexpr (PAIR) {
          mma_bf16_pair(d, ad, bd, idesc, accumulate | (k > 0));
        } else {
          mma_bf16(d, ad, bd, idesc, accumulate | (k > 0));
        }
      };
      if (left >= BK) {
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) mma(k);
      } else {
        for (int k = 0; 16 * k < left; ++k) mma(k);  // behind K's end there are zeros
      }
      accumulate = 1;
      any = true;
      if constexpr (PAIR) {
        mma_commit_pair_both(&s.empty[stage]);
      } else {
        mma_commit(&s.empty[stage]);
      }
      if (++stage == stages) {
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

// Of two warps.
__device__ __forceinline__ void meet(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool both(int id, bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(mine)), "r"(id)
      : "memory");
  return all != 0;
}

template <bool PAIR, bool GATED>
__device__ __forceinline__ void epilogue_loop(const LinArgs& a, const Shared& s, uint32_t tmem, int warp) {
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int lane = static_cast<int>(lane_id());
  const int quarter = warp & 3, phase_of = (warp - 2) >> 2;
  // gated: lanes 0 to 63 are the gate's rows, the others the up projection's
  const int up = GATED ? quarter >> 1 : 0;
  const int lanes = GATED ? (quarter & 1) * 32 : quarter * 32;
  // a warp's buffer, and that of the one with the same rows of the other weight
  float* const mine = s.swap + ((quarter * PHASES) + phase_of) * (SWAP_BYTES / 4) + lane;
  float* const other = s.swap + (((quarter ^ 2) * PHASES) + phase_of) * (SWAP_BYTES / 4) + lane;
  const int barrier = 1 + (quarter & 1) * PHASES + phase_of;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t release = PAIR ? mapa_shared(smem_u32(s.acc_empty), 0) : smem_u32(s.acc_empty);
  int acc = 0, flip = 0;
  uint32_t acc_phase = 0;
  for (int item = unit; item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const int i = (t.it * (PAIR ? 2 : 1) + rank) * (GATED ? LIN_BI / 2 : LIN_BI) + lanes + lane;
    const bool inside = i < p.I;
    const float bias = p.e.bias && p.splits == 1 && inside ? load_scalar(p.e.bias, p.e.bias_type, i) : 0.0f;
    bool ok = true;
    if (lane == 0) ok = wait_bounded_long(&s.acc_full[acc], acc_phase, s.abort_flag, &linear_error);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if constexpr (GATED) ok = both(barrier, ok);  // where a wait ran out, neither waits for the other any more
    if (!ok) break;
    tc_fence_after();
    const uint32_t from = lane_base + static_cast<uint32_t>(acc * ACC_COLS);
    for (int c = phase_of; c < p.jt / CHUNK; c += PHASES) {
      const int j0 = t.jt * p.jt + CHUNK * c;
      const int n = min(CHUNK, p.J - j0);
      if (n <= 0) break;  // the same in all lanes, and in both warps of a gated exchange
      uint32_t r[CHUNK];
      Residual<CHUNK> res;
      if (!GATED && p.e.res && p.splits == 1 && inside) res.load(p.e, i, j0, n);
      __syncwarp();  // the lanes outside of the matrix are back
      tmem_ld16(from + CHUNK * c, r);
      tmem_ld_wait();
      if (p.splits > 1) {  // a partial sum
        if (!inside) continue;
        float z[CHUNK];
#pragma unroll
        for (int u = 0; u < CHUNK; ++u) z[u] = __uint_as_float(r[u]);
        put_rows32(p.part, p.I, (static_cast<int64_t>(t.split * (GATED ? 2 : 1) + up) * p.J + j0) * p.I + i, z, n);
      } else if constexpr (GATED) {
        // the gate's warp finishes the first half of the columns, the other the second
        float* const give = mine + flip * HALF * 32;
        const float* const take = other + flip * HALF * 32;
#pragma unroll
        for (int u = 0; u < HALF; ++u) give[u * 32] = __uint_as_float(up ? r[u] : r[HALF + u]);
        meet(barrier);
        float z0[HALF], z1[HALF];
#pragma unroll
        for (int u = 0; u < HALF; ++u) {
          const float own = __uint_as_float(up ? r[HALF + u] : r[u]), got = take[u * 32];
          z0[u] = up ? got : own;
          z1[u] = up ? own : got;
        }
        flip ^= 1;  // the other warp has read this buffer before it meets the next barrier
        const int left = n - up * HALF;
        if (inside && left > 0) finish_column<true>(p.e, a.bf16, 0.0f, i, j0 + up * HALF, left, z0, z1, Residual<HALF>{});
      } else if (inside) {
        float z[CHUNK];
#pragma unroll
        for (int u = 0; u < CHUNK; ++u) z[u] = __uint_as_float(r[u]);
        finish_column<false>(p.e, a.bf16, bias, i, j0, n, z, z, res);
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
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
    for (int i = 0; i < a.stages; ++i) {
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
    if (lane_id() == 0) mma_loop<PAIR>(a, s, tmem);
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
  return cudaFuncSetAttribute(linear_kernel<PAIR, GATED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              shared_bytes<GATED>());
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
  cfg.dynamicSmemBytes = shared_bytes<true>();
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, linear_kernel<true, true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_linear_gemm(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(pair ? 2 * units : units)), block(THREADS);
  const unsigned cluster = pair ? 2 : 1;
  if (pair) {
    return gated ? launch_after(linear_kernel<true, true>, grid, block, shared_bytes<true>(), cluster, s, a)
                 : launch_after(linear_kernel<true, false>, grid, block, shared_bytes<false>(), cluster, s, a);
  }
  return gated ? launch_after(linear_kernel<false, true>, grid, block, shared_bytes<true>(), cluster, s, a)
               : launch_after(linear_kernel<false, false>, grid, block, shared_bytes<false>(), cluster, s, a);
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

// Persistent, warp-specialised tcgen05 GEMM of the layers in front of the head:
//
//   out[j][i] = epilogue(sum over k of A(i, k) B(j, k))
//
// A holds what becomes the contiguous index of the output (weights in the
// forward pass, so that few tokens make narrow tiles and not empty MMA rows, and a
// thread of the epilogue keeps its four biases in registers), B its rows (tokens).  Either may
// be stored with k contiguous or with its own index contiguous:
//
//   forward          A = W  [N, K] along k       B = x  [M, K] along k
//   dx = dz W        A = W  [N, K] along i = K   B = dz [M, N] along k = N
//   dW = dz^T x      A = x  [M, K] along i = K   B = dz [M, N] along j = N
//
// Up to three products run in one launch (dx and both dW of a gated layer); dx of a
// gated layer is one sum over two pairs of operands.  A gated forward's 128 MMA
// rows are 64 of each weight in turns of 16, so that its loads and MMAs are those of a
// layer twice as wide, and a thread of the epilogue has both values of an output.
//
// Roles (384 threads): lane 0 of warp 0 loads A, that of warp 10 B (TMA; a pair's stages
// are 128 deep in K, a single CTA's 64, as many as fit in 192 KiB; one thread for both
// needed 560 of a stage's 950 cycles: 16,384 x 2,048 x 4,096 took 161 us and not 155),
// warp 1 issues tcgen05.mma into one of two TMEM accumulators (the whole warp runs the
// loop, one elected lane the instruction: its operands stay uniform, and a stage of a narrow
// tile takes 760 cycles; on a path of one lane it took 950), warps 2 to 9
// are the epilogue (warp w reads TMEM lanes 32 (w % 4) to + 31, and every second 32
// columns), and warp 11 adds up the parts of a bias's gradient where there are some.
// CTA pairs share an MMA of M = 256: each CTA holds 128 rows of A and half of B's
// columns.
//
// The epilogue reads the accumulator in the layout of matrix fragments, so that 16-bit
// results pass through shared memory by transposing matrix stores and leave in vectors of
// 16 bytes: with a store of 2 bytes a thread and value a tile of 128 x 256 took 3.7 us,
// longer than its MMAs where K is short, and 8,192 x 896 x 4,864 49 us and not 44.
// Results whose rows are off 16 bytes and fp32 ones are stored directly, 8 values of a
// row together.
//
// Bound by the tensor cores for many rows: 65,536 x 2,048 x 8,192 with bias and gelu
// 1.39 ms (1.58 PFLOP/s), 8,192 x 9,216 x 2,304 193 us (1.80), 16,384 x 2,048 x 4,096
// 153 us (1.80); where K is short by the epilogue, 8,192 x 896 x 4,864 44 us (1.63).  A
// launch costs some 5 us beside its products: 128 x 896 x 896 takes 5.8 us.  Narrow tiles
// are bound by the MMAs' reading 128 rows of A from shared memory.
#pragma once

#include "gemm_args.h"
#include "internal.h"
#include "linear.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace cce {
namespace lin {

constexpr int EPI_WARPS = 8;
constexpr int PHASES = EPI_WARPS / 4;  // warps that share the columns of 32 TMEM lanes
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int ACC_COLS = 256;  // TMEM columns of one of the two accumulators
constexpr int CHUNK = 32;           // columns of a warp at a time
constexpr int GROUP = 64 * 128;  // bytes of 64 rows of 128 bytes
constexpr int TURN = LIN_TURN;
constexpr int STAGING = 32 * CHUNK * 2;  // a warp's tile
constexpr int BAR_BYTES_LIN = 512;

constexpr int SHARED = 1024 + LIN_RING_BYTES + EPI_WARPS * STAGING + BAR_BYTES_LIN;
static_assert(SHARED <= 227 * 1024, "shared memory of a CTA");

struct Shared {
  uint8_t* ring;
  uint64_t* full;       // [LIN_MAX_STAGES]
  uint64_t* empty;      // [LIN_MAX_STAGES]
  uint64_t* acc_full;   // [2]
  uint64_t* acc_empty;  // [2]
  uint64_t* drain;
  uint32_t* tmem;
  int* abort_flag;
  uint8_t* staging;  // [EPI_WARPS][STAGING]
};

__device__ __forceinline__ Shared carve(uint8_t* raw) {
  Shared s;
  s.ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  s.staging = s.ring + LIN_RING_BYTES;
  s.full = reinterpret_cast<uint64_t*>(s.staging + EPI_WARPS * STAGING);
  s.empty = s.full + LIN_MAX_STAGES;
  s.acc_full = s.empty + LIN_MAX_STAGES;
  s.acc_empty = s.acc_full + 2;
  s.drain = s.acc_empty + 2;
  s.tmem = reinterpret_cast<uint32_t*>(s.drain + 1);
  s.abort_flag = reinterpret_cast<int*>(s.tmem + 1);
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

// The fields' lines of the constant cache, and a tile's numbers: they have to be there behind this.
__device__ __forceinline__ void touch(const LinProblem& p, const Tile& t) {
  asm volatile("" ::"r"(t.it), "r"(t.jt), "r"(t.kb), "r"(t.kb_end), "r"(p.I), "r"(p.klen[0]), "r"(p.jt), "r"(p.wide),
               "l"(p.e.y), "l"(p.e.res), "r"(p.e.act));
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
  // Gated: 64 rows of each weight from i0 on, in turns.
  __device__ __forceinline__ void turns(const LinProblem& p, uint8_t* to, int i0, int k0) const {
#pragma unroll
    for (int k = 0; k < lin_bk(PAIR); k += 64, to += 2 * GROUP) {
      if (p.a_4d) {
        if constexpr (PAIR) {
          tma_load_4d_pair(&p.a[0], lead, to, k0 + k, 0, 0, i0 / TURN);
        } else {
          tma_load_4d(&p.a[0], bar, to, k0 + k, 0, 0, i0 / TURN);
        }
      } else {
        for (int r = 0; r < 2 * LIN_BI / 2 / TURN; ++r) box2(&p.a[r & 1], to + r * TURN * 128, k0 + k, i0 + (r >> 1) * TURN);
      }
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

// The loads of A, whose thread announces the bytes of both, or of B.
template <bool PAIR, bool GATED, bool A>
__device__ __forceinline__ void load_loop(const LinArgs& a, const Shared& s, const Tile& first) {
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
  Tile next = first;
  for (int item = unit; ok && item < a.items; item += units) {
    const Tile t = next;
    const LinProblem& p = *t.p;
    const int kb_first = p.kb_first;
    const bool mn = A ? p.a_mn : p.b_mn, whole = A ? p.a_3d : p.b_3d;
    const int rows = PAIR ? p.jt / 2 : p.jt;
    const int loaded = lin_b_rows(p.jt, PAIR, p.b_mn);
    const int i0 = (t.it * (PAIR ? 2 : 1) + rank) * (GATED ? LIN_BI / 2 : LIN_BI);
    const int j0 = t.jt * p.jt + rank * rows;
    const uint32_t bytes = static_cast<uint32_t>((A_BYTES + loaded * BK * 2) * (PAIR ? 2 : 1));
    for (int kb = t.kb; kb < t.kb_end; ++kb) {
      if (!wait_bounded_long(&s.empty[stage], phase ^ 1u, abort_flag, a.error)) {
        ok = false;
        break;
      }
      const Loader<PAIR> load{&s.full[stage], lead + 8u * static_cast<uint32_t>(stage)};
      uint8_t* to = s.ring + stage * stage_bytes;
      if (A && rank == 0) mbar_arrive_expect_tx(&s.full[stage], bytes);
      const int part = !GATED && kb >= kb_first ? 1 : 0;
      const int k0 = (part ? kb - kb_first : kb) * BK;
      if constexpr (!A) {
        load.operand(&p.b[part], mn, whole, to + A_BYTES, j0, rows, k0, rows * 128);
      } else if constexpr (GATED) {
        load.turns(p, to, i0, k0);
      } else {
        load.operand(&p.a[part], mn, whole, to, i0, LIN_BI, k0, 2 * GROUP);
      }
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
      if (kb == t.kb && item + units < a.items) next = tile_of(a, item + units);
    }
  }
  if (ok && !*abort_flag) {
    // a pair's stages are handed back by the even CTA's MMAs: this CTA stays until all of them have been
    for (int i = 0; A && PAIR && i < stages; ++i) {
      if (!wait_bounded_long(&s.empty[stage], phase ^ 1u, abort_flag, a.error)) break;
      if (++stage == stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    return;
  }
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

// PARTS, here and below: results whose sum goes on in another accumulator every LIN_CHUNK_K (in kernels of their own: as a
// choice at run time it cost the others 0.3 to 0.7 us a launch).
template <bool PAIR, bool PARTS>
__device__ __forceinline__ void mma_loop(const LinArgs& a, const Shared& s, uint32_t tmem, const Tile& first) {
  if (PAIR && cluster_ctarank() != 0) return;  // the even CTA issues for both
  constexpr int BK = lin_bk(PAIR), A_BYTES = LIN_BI * BK * 2;
  volatile int* abort_flag = s.abort_flag;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int stages = a.stages, stage_bytes = a.stage_bytes;
  int stage = 0, acc = 0;
  uint32_t phase = 0, acc_phase = 0;
  bool any = false, ok = true;
  const uint32_t lead = elect_lane();
  // parts of K, and whether they take the accumulators in turn
  const int chunk = PARTS ? a.chunk : 1 << 30, other = PARTS ? 0 : 1;
  // (the divisions for the next tile are made while this one's MMAs run: some 700 cycles between two tiles otherwise)
  Tile next = first;
  for (int item = unit; ok && item < a.items; item += units) {
    const Tile t = next;
    const LinProblem& p = *t.p;
    const bool a_mn = p.a_mn, b_mn = p.b_mn;
    const int kb_first = p.kb_first, klen0 = p.klen[0], klen1 = p.klen[1];
    // bits 7-9 and 10-12 of the descriptor: 1 = bf16, 0 = fp16
    const uint32_t idesc = idesc_bf16(PAIR ? 2 * LIN_BI : LIN_BI, p.jt, a_mn, b_mn) & (a.bf16 ? ~0u : ~((1u << 7) | (1u << 10)));
    // along its own index: 64-element groups of BK rows of 128 bytes, 16 of k are 16 rows; along
    // k: 16 of k are 32 bytes of a row, 64 of k all rows
    const uint32_t a_lbo = a_mn ? BK * 128u : 16u, b_lbo = b_mn ? BK * 128u : 16u;
    const uint32_t a_step = (a_mn ? 2048u : 32u) >> 4, b_step = (b_mn ? 2048u : 32u) >> 4;
    const uint32_t a_next = (a_mn ? 8192u : 2u * GROUP) >> 4;
    const uint32_t b_next = (b_mn ? 8192u : (PAIR ? p.jt / 2 : p.jt) * 128u) >> 4;
    for (int from = t.kb; from < t.kb_end; from += chunk) {
      if (!__all_sync(0xffffffffu, wait_bounded_long(&s.acc_empty[acc], acc_phase ^ 1u, abort_flag, a.error))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(acc * ACC_COLS);
      uint32_t accumulate = 0;
      const int part_end = min(from + chunk, t.kb_end);
      for (int kb = from; kb < part_end; ++kb) {
        if (!__all_sync(0xffffffffu, wait_bounded_long(&s.full[stage], phase, abort_flag, a.error))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int left = kb < kb_first ? klen0 - kb * BK : klen1 - (kb - kb_first) * BK;
        const uint32_t at = smem_u32(s.ring + stage * stage_bytes);
        const uint64_t a_desc = smem_desc_sw128(at, a_lbo, 1024u);
        const uint64_t b_desc = smem_desc_sw128(at + A_BYTES, b_lbo, 1024u);
        const auto mma = [&](int k) {
          const uint64_t ad = a_desc + (k >> 2) * a_next + (k & 3) * a_step, bd = b_desc + (k >> 2) * b_next + (k & 3) * b_step;
          if constexpr (PAIR) {
            mma_bf16_pair_by(lead, d, ad, bd, idesc, accumulate | (k > 0));
          } else {
            mma_bf16_by(lead, d, ad, bd, idesc, accumulate | (k > 0));
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
        if (lead) {
          if constexpr (PAIR) {
            mma_commit_pair_both(&s.empty[stage]);
          } else {
            mma_commit(&s.empty[stage]);
          }
        }
        __syncwarp();
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
        if (kb == t.kb && item + units < a.items) next = tile_of(a, item + units);
      }
      if (!ok) break;
      if (lead) {
        if constexpr (PAIR) {
          mma_commit_pair_both(&s.acc_full[acc]);
        } else {
          mma_commit(&s.acc_full[acc]);
        }
      }
      __syncwarp();
      acc ^= other;
      if (acc == 0) acc_phase ^= 1u;
    }
    if (!ok) break;
  }
  // and the even one until both CTAs' epilogues have handed back its accumulators
  for (int i = 0; PAIR && ok && i < (PARTS ? 1 : 2); ++i) {
    if (!__all_sync(0xffffffffu, wait_bounded_long(&s.acc_empty[acc], acc_phase ^ 1u, abort_flag, a.error))) break;
    acc ^= 1;
    if (acc == 0) acc_phase ^= 1u;
  }
  if (lead && *abort_flag && any) {
    if constexpr (PAIR) {
      mma_commit_pair_local(s.drain);
    } else {
      mma_commit(s.drain);
    }
    volatile int none = 0;
    wait_bounded(s.drain, 0, &none, nullptr);
  }
}

// A warp has read its part of an accumulator: the values are in registers, so that nothing but the arrival has to reach
// the other CTA.  (With a release the last chunk's stores had to land first: 2,000 cycles a tile.)
template <bool PAIR>
__device__ __forceinline__ void release_accumulator(const Shared& s, int acc, uint32_t lead) {
  tc_fence_before();
  __syncwarp();
  if (lane_id() == 0) {
    if constexpr (PAIR) {
      mbar_arrive_cluster_relaxed(lead + 8u * static_cast<uint32_t>(acc));
    } else {
      mbar_arrive(&s.acc_empty[acc]);
    }
  }
}

// What a thread holds of a chunk's 32 columns j and R x 8 rows i: rows 8 apart of pairs of neighbouring columns, the
// pairs 8 apart, as [pair][row][column of the pair].
template <int R>
struct Fragment {
  float v[8 * R];

  // As 16-bit values to the first n columns and `rows` rows (a multiple of 8) of a matrix whose rows start on 16 bytes;
  // p: the thread's place in it, column lane / R and row 8 (lane % R).  `tile`: 16 R bytes of shared memory for each
  // column, swizzled so that neither access has bank conflicts.
  __device__ __forceinline__ void store_wide(uint32_t tile, uint16_t* p, int64_t pitch, int type, int n, int rows) const {
    const auto place = [&](uint32_t j, uint32_t vector) {
      return tile + j * 16u * R + ((vector ^ (R == 4 ? j >> 1 & 3u : j >> 2 & 1u)) << 4);
    };
    const uint32_t lane = lane_id(), which = lane >> 3;
    const uint32_t to = place(8u * (which / R) + (lane & 7u), which % R), from = place(lane / R, lane % R);
    uint32_t two[4 * R];
    to_bits16(type, v, two);
    __syncwarp();  // what was there has been read
#pragma unroll
    for (int q = 0; q < R; ++q)  // four matrices at a time: 32 / R columns, 512 bytes
      stmatrix_columns(to + 512u * q, two[4 * q], two[4 * q + 1], two[4 * q + 2], two[4 * q + 3]);
    __syncwarp();
    uint4 w[R];
#pragma unroll
    for (int q = 0; q < R; ++q)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[q].x), "=r"(w[q].y), "=r"(w[q].z), "=r"(w[q].w)
                   : "r"(from + 512u * q)
                   : "memory");
    const int j = static_cast<int>(lane) / R;
    if (8 * (static_cast<int>(lane) % R) >= rows) n = 0;
#pragma unroll
    for (int q = 0; q < R; ++q, p += 32 / R * pitch) {
      if (q * (32 / R) + j < n) *reinterpret_cast<uint4*>(p) = w[q];
    }
  }
  // To the first n columns and `rows` rows of a matrix, whose element of the thread's first place is at p.
  __device__ __forceinline__ void store(float* p, int64_t pitch, int n, int rows) const {
    store_each<float>(p, pitch, n, rows, [&](int x) { return v[x]; });
  }
  __device__ __forceinline__ void store(uint16_t* p, int64_t pitch, int type, int n, int rows) const {
    uint32_t two[4 * R];
    to_bits16(type, v, two);
    store_each<uint16_t>(p, pitch, n, rows, [&](int x) { return static_cast<uint16_t>(two[x / 2] >> (16 * (x & 1))); });
  }

 private:
  template <typename T, typename Value>
  __device__ __forceinline__ void store_each(T* p, int64_t pitch, int n, int rows, Value value) const {
    const int c0 = 2 * static_cast<int>(lane_id() & 3u), r0 = static_cast<int>(lane_id() >> 2);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        T* row = p + (8 * b + c) * pitch;
        if (8 * b + c0 + c >= n) continue;
#pragma unroll
        for (int m = 0; m < R; ++m) {
          if (r0 + 8 * m < rows) row[8 * m] = value(2 * R * b + 2 * m + c);
        }
      }
    }
  }
};

// The residual's values of a chunk as they are in memory, loaded ahead of what they are added to.
struct Residuals {
  uint32_t raw[32];

  // p: the thread's first place in a row; j: its first row.
  template <typename T>
  __device__ __forceinline__ void load(const T* p, const LinEpilogue& e, int64_t j, int n, int rows) {
    if (e.res_inner == 0) {
      const int64_t pitch = e.res_pitch;
      p += j * pitch;
      load_rows(n, rows, [&](int x) { return p + x * pitch; });
    } else {
      load_rows(n, rows, [&](int x) { return p + res_row(e, j + x); });
    }
  }
  template <typename Row>
  __device__ __forceinline__ void load_rows(int n, int rows, Row row_of) {
    const int c0 = 2 * static_cast<int>(lane_id() & 3u), r0 = static_cast<int>(lane_id() >> 2);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const auto row = row_of(8 * b + c);
#pragma unroll
        for (int m = 0; m < 4; ++m)
          raw[8 * b + 2 * m + c] = 8 * b + c0 + c < n && r0 + 8 * m < rows ? row[8 * m] : 0;
      }
    }
  }
  __device__ __forceinline__ void add_to(Fragment<4>& f, bool y32, bool bf16) const {
    if (y32) {
#pragma unroll
      for (int e = 0; e < 32; ++e) f.v[e] += __uint_as_float(raw[e]);
    } else if (bf16) {
#pragma unroll
      for (int e = 0; e < 32; ++e) f.v[e] += __uint_as_float(raw[e] << 16);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) f.v[e] += __half2float(__ushort_as_half(static_cast<uint16_t>(raw[e])));
    }
  }
};

// A chunk of the accumulator as it comes from TMEM: lanes 0 to 15 and 16 to 31 of a warp's quarter (gated: the gate's
// and the up projection's).
struct Chunk {
  uint32_t lo[16], hi[16];

  __device__ __forceinline__ void load(uint32_t first, uint32_t second) {
    tmem_ld_16x256(first, lo);
    tmem_ld_16x256(second, hi);
  }
  __device__ __forceinline__ void wait() {
    tmem_ld_wait16(lo);
    tmem_ld_wait16(hi);
  }
  // To what there is, the sum so far at those places is added.
  __device__ __forceinline__ void add(uint32_t first, uint32_t second) {
    add_half(first, lo);
    add_half(second, hi);
  }
  __device__ __forceinline__ void store(uint32_t first, uint32_t second) const {
    tmem_st_16x256(first, lo);
    tmem_st_16x256(second, hi);
  }
  __device__ __forceinline__ static void add_half(uint32_t at, uint32_t (&to)[16]) {
    uint32_t so_far[16];
    tmem_ld_16x256(at, so_far);
    tmem_ld_wait16(so_far);
#pragma unroll
    for (int x = 0; x < 16; ++x) to[x] = __float_as_uint(__uint_as_float(so_far[x]) + __uint_as_float(to[x]));
  }
  __device__ __forceinline__ void get(Fragment<4>& f) const {
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        f.v[8 * b + x] = __uint_as_float(lo[4 * b + x]);
        f.v[8 * b + 4 + x] = __uint_as_float(hi[4 * b + x]);
      }
  }
  __device__ __forceinline__ void get(Fragment<2>& gate, Fragment<2>& up) const {
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      gate.v[x] = __uint_as_float(lo[x]);
      up.v[x] = __uint_as_float(hi[x]);
    }
  }
};

// A warp's share of a tile: `rows` rows i from i0 on, and chunks of 32 of the `cols` columns from j0 on, PHASES apart.
struct Share {
  int i0, j0, rows, cols, chunks;
  uint32_t first, second;  // where chunk 0 is in TMEM, its halves
  uint32_t total;          // the sum of K's parts before this one, so far behind them; 0: there is none
  uint32_t tile;           // of the warp in shared memory
  float bias[4];
};

// Wide results of the accumulator alone, for gated layers with the values in front of the activation (KEEP) or without: the
// next chunk comes while one is finished.  (4,096 x 4,864 x 896 with them took 57 us by finish_any and 54 so.  Layers without
// a gate hold twice the values of one matrix: their registers ran out, 42 us became 50.)
template <bool PAIR, bool GATED, int ACT, bool KEEP>
__device__ __forceinline__ void finish_lean(const Shared& s, const Share& w, const LinEpilogue& e, int type, int acc,
                                            uint32_t release) {
  constexpr int R = GATED ? 2 : 4;
  const int lane = static_cast<int>(lane_id());
  const int64_t pitch = e.y_pitch;
  uint16_t* y = static_cast<uint16_t*>(e.y) + static_cast<int64_t>(w.j0 + lane / R) * pitch + w.i0 + 8 * (lane % R);
  const int64_t z_pitch = e.z_pitch;
  int64_t z = static_cast<int64_t>(w.j0 + lane / R) * z_pitch + w.i0 + 8 * (lane % R);
  const auto keep = [&](const Fragment<2>& f, void* to, int n) {
    f.store_wide(w.tile, static_cast<uint16_t*>(to) + z, z_pitch, e.z_type, n, w.rows);
  };
  int n = w.cols;
  const auto step = [&](Chunk& now, Chunk& next, int c) {
    now.wait();
    if (c + 1 < w.chunks) {
      next.load(w.first + CHUNK * PHASES * (c + 1), w.second + CHUNK * PHASES * (c + 1));
    } else {
      release_accumulator<PAIR>(s, acc, release);
    }
    if constexpr (GATED) {
      Fragment<2> gate, up;
      now.get(gate, up);
      if (KEEP) {
        keep(gate, e.z[0], n);
        keep(up, e.z[1], n);
      }
      activate_as<ACT>(gate.v);
#pragma unroll
      for (int x = 0; x < 16; ++x) gate.v[x] *= up.v[x];
      gate.store_wide(w.tile, y, pitch, type, n, w.rows);
    } else {
      Fragment<4> f;
      now.get(f);
#pragma unroll
      for (int x = 0; x < 32; ++x) f.v[x] += w.bias[x >> 1 & 3];
      activate_as<ACT>(f.v);
      f.store_wide(w.tile, y, pitch, type, n, w.rows);
    }
    y += CHUNK * PHASES * pitch;
    z += CHUNK * PHASES * z_pitch;
    n -= CHUNK * PHASES;
  };
  Chunk a, b;
  a.load(w.first, w.second);
  for (int c = 0; c < w.chunks; c += 2) {
    step(a, b, c);
    if (c + 1 < w.chunks) step(b, a, c + 1);
  }
}

// Everything else: a residual, a layer's values in front of its activation, fp32 results and ones off 16 bytes.
template <bool PAIR, bool GATED, int ACT, bool PARTS>
__device__ __forceinline__ void finish_any(const Shared& s, const Share& w, const LinEpilogue& e, bool wide, int type,
                                           int acc, uint32_t release) {
  constexpr int R = GATED ? 2 : 4;
  const int lane = static_cast<int>(lane_id());
  const bool y32 = !GATED && e.y_type == CCE_F32, has_z = e.z[0] != nullptr, has_res = !GATED && e.res;
  // the thread's first place of a chunk: as one of fragments, and of wide stores
  const int64_t wide_y = static_cast<int64_t>(w.j0 + lane / R) * e.y_pitch + w.i0 + 8 * (lane % R);
  const int64_t wide_z = static_cast<int64_t>(w.j0 + lane / R) * e.z_pitch + w.i0 + 8 * (lane % R);
  const int64_t ti = w.i0 + lane / 4, tj = w.j0 + 2 * (lane & 3);
  for (int c = 0; c < w.chunks; ++c) {
    const int jc = CHUNK * PHASES * c, n = w.cols - jc;
    Chunk chunk;
    chunk.load(w.first + jc, w.second + jc);
    Residuals res;
    if (has_res) {
      if (y32) {
        res.load(static_cast<const uint32_t*>(e.res) + ti, e, tj + jc, n, w.rows);
      } else {
        res.load(static_cast<const uint16_t*>(e.res) + ti, e, tj + jc, n, w.rows);
      }
    }
    chunk.wait();
    if (PARTS && w.total) chunk.add(w.first + w.total + jc, w.second + w.total + jc);
    if (c + 1 == w.chunks) {
      release_accumulator<PAIR>(s, acc, release);
    } else {
      __syncwarp();
    }
    const auto put = [&](const Fragment<R>& f, void* to, int64_t wide_at, int64_t pitch, int as) {
      if (wide) {
        f.store_wide(w.tile, static_cast<uint16_t*>(to) + wide_at + jc * pitch, pitch, as, n, w.rows);
      } else {
        f.store(static_cast<uint16_t*>(to) + (tj + jc) * pitch + ti, pitch, as, n, w.rows);
      }
    };
    if constexpr (GATED) {
      Fragment<2> gate, up;
      chunk.get(gate, up);
      if (has_z) {
        put(gate, e.z[0], wide_z, e.z_pitch, e.z_type);
        put(up, e.z[1], wide_z, e.z_pitch, e.z_type);
      }
      activate_as<ACT>(gate.v);
#pragma unroll
      for (int x = 0; x < 16; ++x) gate.v[x] *= up.v[x];
      put(gate, e.y, wide_y, e.y_pitch, type);
    } else {
      Fragment<4> f;
      chunk.get(f);
#pragma unroll
      for (int x = 0; x < 32; ++x) f.v[x] += w.bias[x >> 1 & 3];
      if (has_z) put(f, e.z[0], wide_z, e.z_pitch, e.z_type);
      activate_as<ACT>(f.v);
      if (has_res) res.add_to(f, y32, type == BITS_BF16);
      if (y32) {
        f.store(static_cast<float*>(e.y) + (tj + jc) * e.y_pitch + ti, e.y_pitch, n, w.rows);
      } else {
        put(f, e.y, wide_y, e.y_pitch, type);
      }
    }
  }
}

// Partial sums of a split of K.
template <bool PAIR, bool GATED, bool PARTS>
__device__ __forceinline__ void store_partial(const Shared& s, const Share& w, const LinProblem& p, int split, int acc,
                                              uint32_t release) {
  const int lane = static_cast<int>(lane_id());
  const int64_t mats = GATED ? 2 : 1;
  float* to = p.part + (mats * split * p.J + w.j0 + 2 * (lane & 3)) * p.I + w.i0 + lane / 4;
  for (int c = 0; c < w.chunks; ++c, to += static_cast<int64_t>(CHUNK * PHASES) * p.I) {
    const int jc = CHUNK * PHASES * c, n = w.cols - jc;
    Chunk chunk;
    chunk.load(w.first + jc, w.second + jc);
    chunk.wait();
    if (PARTS && w.total) chunk.add(w.first + w.total + jc, w.second + w.total + jc);
    if (c + 1 == w.chunks) {
      release_accumulator<PAIR>(s, acc, release);
    } else {
      __syncwarp();
    }
    if constexpr (GATED) {
      Fragment<2> gate, up;
      chunk.get(gate, up);
      gate.store(to, p.I, n, w.rows);
      up.store(to + static_cast<int64_t>(p.J) * p.I, p.I, n, w.rows);
    } else {
      Fragment<4> f;
      chunk.get(f);
      f.store(to, p.I, n, w.rows);
    }
  }
}

// A part of K that others follow, to the sum so far.
template <bool PAIR>
__device__ __forceinline__ void add_to_total(const Shared& s, const Share& w, bool none_yet, int acc, uint32_t release) {
  for (int c = 0; c < w.chunks; ++c) {
    const int jc = CHUNK * PHASES * c;
    const uint32_t first = w.first + ACC_COLS + jc, second = w.second + ACC_COLS + jc;
    Chunk chunk;
    chunk.load(w.first + jc, w.second + jc);
    chunk.wait();
    if (!none_yet) chunk.add(first, second);
    chunk.store(first, second);
  }
  tmem_st_wait();
  release_accumulator<PAIR>(s, acc, release);
}

template <bool PAIR, bool GATED, int ACT, bool PARTS>
__device__ __forceinline__ void epilogue_loop(const LinArgs& a, const Shared& s, uint32_t tmem, int warp) {
  constexpr int ROWS = GATED ? TURN : 32;  // of the output, a warp
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int unit = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int units = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);
  const int lane = static_cast<int>(lane_id());
  const int quarter = warp & 3, phase_of = (warp - 2) >> 2;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t release = PAIR ? mapa_shared(smem_u32(s.acc_empty), 0) : smem_u32(s.acc_empty);
  const int type = a.bf16 ? BITS_BF16 : BITS_F16;
  Share w;
  w.tile = smem_u32(s.staging + (quarter * PHASES + phase_of) * STAGING);
  int acc = 0;
  uint32_t acc_phase = 0;
  for (int item = unit; item < a.items; item += units) {
    const Tile t = tile_of(a, item);
    const LinProblem& p = *t.p;
    const LinEpilogue& e = p.e;
    w.i0 = (t.it * (PAIR ? 2 : 1) + rank) * (GATED ? LIN_BI / 2 : LIN_BI) + quarter * ROWS;
    w.j0 = t.jt * p.jt + CHUNK * phase_of;
    w.rows = p.I - w.i0;
    w.cols = p.J - w.j0;
    w.chunks = min((p.jt / CHUNK - phase_of + PHASES - 1) / PHASES, (w.cols + CHUNK * PHASES - 1) / (CHUNK * PHASES));
    const bool whole = p.splits == 1, wide = p.wide;
    if constexpr (!GATED) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int i = lane / 4 + 8 * m;
        w.bias[m] = whole && e.bias && i < w.rows ? load_scalar(e.bias, e.bias_type, w.i0 + i) : 0.0f;
      }
    }
    w.first = w.second = lane_base + static_cast<uint32_t>(acc * ACC_COLS + CHUNK * phase_of);
    (GATED && p.up_first ? w.first : w.second) += 16u << 16;
    const auto filled = [&] {
      bool ok = true;
      if (lane == 0) ok = wait_bounded_long(&s.acc_full[acc], acc_phase, s.abort_flag, a.error);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      tc_fence_after();
      return ok;
    };
    w.total = 0;
    bool ok = true;
    if constexpr (PARTS) {
      // parts of K one after the other in the first accumulator, their sum in the second one's place
      for (int kb = t.kb; kb + a.chunk < t.kb_end; kb += a.chunk) {
        ok = filled();
        if (!ok) break;
        add_to_total<PAIR>(s, w, kb == t.kb, acc, release);
        acc_phase ^= 1u;
        w.total = ACC_COLS;
      }
    }
    if (!ok || !filled()) break;
    if (w.chunks <= 0) {
      release_accumulator<PAIR>(s, acc, release);
    } else if (!whole) {
      store_partial<PAIR, GATED, PARTS>(s, w, p, t.split, acc, release);
    } else if (wide && !e.z[0] && !e.res) {
      finish_lean<PAIR, GATED, ACT, false>(s, w, e, type, acc, release);
    } else if (GATED && wide) {
      finish_lean<PAIR, GATED, ACT, GATED>(s, w, e, type, acc, release);
    } else {
      finish_any<PAIR, GATED, ACT, PARTS>(s, w, e, wide, type, acc, release);
    }
    if (PARTS) {
      acc_phase ^= 1u;
    } else {
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
}

template <bool PAIR, bool GATED, int ACT, bool PARTS>
__global__ void __launch_bounds__(THREADS, 1) linear_kernel(const __grid_constant__ LinArgs a) {
  extern __shared__ uint8_t raw[];
  const Shared s = carve(raw);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
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
  if (warp == 0 && lane_id() < 2 * a.problems) {  // before the first copies need them
    const LinProblem& p = a.p[lane_id() >> 1];
    tma_prefetch_desc(lane_id() & 1 ? &p.b[0] : &p.a[0]);
    if (GATED || p.klen[1] > 0) tma_prefetch_desc(lane_id() & 1 ? &p.b[GATED ? 0 : 1] : &p.a[1]);
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
  // what the first tile needs of the arguments is read, and its divisions are made, while the kernel before still runs
  const Tile first = tile_of(a, PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x));
  touch(*first.p, first);
  wait_for_previous();

  if (warp == 0) {
    if (lane_id() == 0) load_loop<PAIR, GATED, true>(a, s, first);
  } else if (warp == 1) {
    mma_loop<PAIR, PARTS>(a, s, tmem, first);
  } else if (warp == 2 + EPI_WARPS) {
    if (lane_id() == 0) load_loop<PAIR, GATED, false>(a, s, first);
  } else if (warp == 3 + EPI_WARPS) {
    if (a.sum.parts > 0) {
      for (int c = static_cast<int>(blockIdx.x) * 32; c < a.sum.N; c += static_cast<int>(gridDim.x) * 32)
        sum_columns(a.sum, c + static_cast<int>(lane_id()));
    }
  } else {
    epilogue_loop<PAIR, GATED, ACT, PARTS>(a, s, tmem, warp);
  }

  tc_fence_before();
  __syncthreads();
  // no CTA leaves while the other may still signal its barriers: what is signalled has arrived (load_loop and mma_loop
  // end with waits for it), unless a wait ran out
  if constexpr (PAIR) {
    if (*s.abort_flag) {
      cluster_sync();
    } else {
      cluster_sync_relaxed();
    }
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) {
      tmem_dealloc_pair(tmem, TMEM_COLS);
    } else {
      tmem_dealloc(tmem, TMEM_COLS);
    }
  }
}

// The kernels of one activation.
template <int ACT>
cudaError_t prepare() {
  const auto set = [](auto kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SHARED);
  };
  cudaError_t e = set(linear_kernel<false, false, ACT, false>);
  if (e == cudaSuccess) e = set(linear_kernel<false, true, ACT, false>);
  if (e == cudaSuccess) e = set(linear_kernel<true, false, ACT, false>);
  if (e == cudaSuccess) e = set(linear_kernel<true, true, ACT, false>);
  if (e == cudaSuccess) e = set(linear_kernel<false, false, ACT, true>);
  if (e == cudaSuccess) e = set(linear_kernel<true, false, ACT, true>);
  return e;
}

template <int ACT>
cudaError_t launch(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(pair ? 2 * units : units)), block(THREADS);
  const auto with = [&](auto kernel) { return launch_after(kernel, grid, block, SHARED, pair ? 2u : 1u, s, a); };
  if (a.chunk > 0) return pair ? with(linear_kernel<true, false, ACT, true>) : with(linear_kernel<false, false, ACT, true>);
  if (pair) return gated ? with(linear_kernel<true, true, ACT, false>) : with(linear_kernel<true, false, ACT, false>);
  return gated ? with(linear_kernel<false, true, ACT, false>) : with(linear_kernel<false, false, ACT, false>);
}

}  // namespace lin
}  // namespace cce

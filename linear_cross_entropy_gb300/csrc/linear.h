// Products with a fused epilogue (include/cce_layers.h): arguments of the kernels
// and their launchers, shared by the entry points (layers_api.cu), the tcgen05
// GEMM (linear_gemm.cu) and the kernels around it (linear_few.cu, linear_pass.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/cce_layers.h"

namespace cce {

// What happens to an accumulator on its way out: z = acc + bias[i], y = f(z) +
// residual, with [J][I] matrices whose index i is contiguous.  Gated: y = f(z0) z1.
struct LinEpilogue {
  void* y;
  int64_t y_pitch;
  const void* bias;  // [I], may be null
  const void* res;   // of y's type, may be null
  int64_t res_pitch, res_outer;
  int res_inner;  // rows of res at the pitch, such runs res_outer apart; 0: all of them are
  void* z[2];  // pre-activations, may be null
  int64_t z_pitch;
  int y_type, bias_type, act, z_type;  // z_type: the operands', or CCE_KEPT16
};

// out[j][i] = epilogue(sum over k of A(i, k) B(j, k)).  The sum may run over two
// pairs of operands in turn (dx of a gated layer); gated forward: a[0] and a[1]
// are the gate's and the up projection's weights, both against b[0], in turns of 16
// rows (a_4d: one map over both, whichever lies first in memory).
// Tensor maps: an operand whose contiguous extent is a multiple of 64 comes in one
// 3-D box a stage (its groups of 64 as the third dimension), another in 2-D boxes,
// one a group.
struct LinProblem {
  CUtensorMap a[2];
  CUtensorMap b[2];
  int I, J;
  int klen[2];   // elements of either part of the sum (klen[1] = 0: one part)
  int kb_first;  // blocks of K of the first part
  int kb_all;
  int8_t a_mn, b_mn;  // operand stored with its I (J) index contiguous
  int8_t a_3d, b_3d, a_4d, up_first;
  int jt;          // tile width in J
  int i_tiles, j_tiles, splits, kb_split;  // kb_split: blocks of K per split
  int group;       // i tiles that are walked together
  int items;       // i_tiles * j_tiles * splits
  int wide;        // 16-bit results (and no partial sums) whose rows start on 16 bytes, I a multiple of 8
  float* part;     // splits > 1: [splits][GATED ? 2 : 1][J][I]
  LinEpilogue e;
};

// db[c] = the sum over the parts of part[p][c], in a fixed order.
struct LinSum {
  const float* part;
  void* db;
  int parts, N, type;
};

constexpr int LIN_MAX_PROBLEMS = 3;
struct LinArgs {
  LinProblem p[LIN_MAX_PROBLEMS];
  LinSum sum;  // made beside the products (parts = 0: none)
  int problems;
  int items;
  int bf16;  // operands are bf16, else fp16
  int stages, stage_bytes;
  int chunk;  // fp32 results: blocks of K that the tensor core adds up at a time (0: all)
  int32_t* error;  // the device's error word (CCE_DEVERR_*)
};

constexpr int LIN_SMS = 152;  // what sizes of grids and workspaces count with, on any device
constexpr int LIN_BI = 128;  // rows of the MMA a CTA: I extent of a tile (gated: 64 of each weight)
// Blocks of K: a stage's depth.  A pair's loads are issued half as often with the deeper one.
constexpr int lin_bk(bool pair) { return pair ? 128 : 64; }
// Rows of B that a CTA loads for a tile: whole groups of 64 where they are stored along their own index.
__host__ __device__ constexpr int lin_b_rows(int jt, bool pair, bool mn) {
  return mn ? ((pair ? jt / 2 : jt) + 63) / 64 * 64 : pair ? jt / 2 : jt;
}
constexpr int LIN_TURN = 16;  // gated: rows of a weight after which the other's come
constexpr int LIN_RING_BYTES = 192 * 1024;
constexpr int LIN_MAX_STAGES = 10;
// Of an fp32 result the tensor core, which cuts where it could round, adds up so much of K at a time; the epilogue adds
// the parts, to nearest: with K = 9,216 a sum is 1.0e-6 of the norm off and not 1.0e-5, as at K = 1,000, and 8,192 x 9,216 x
// 2,304 takes 245 us and not 197, as both accumulators are taken.  (A 16-bit result's rounding hides what the core cuts, but
// for a relu's slope, which jumps: of 4,096 x 1,024 values of z with K = 9,216 eight had the other sign, one in parts, and the
// gradients were 2.2e-3 of their norm off and not 1.7e-3.  As in any 16-bit product; the time is left to fp32 results.)
constexpr int LIN_CHUNK_K = 1024;

// The launch as `units` persistent CTAs or CTA pairs.
cudaError_t launch_linear_gemm(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s);
cudaError_t launch_linear_gemm_relu(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s);
cudaError_t launch_linear_gemm_gelu(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s);
cudaError_t launch_linear_gemm_gelu_tanh(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s);
cudaError_t launch_linear_gemm_silu(const LinArgs& a, bool pair, bool gated, int units, cudaStream_t s);
cudaError_t prepare_linear_gemm_relu();
cudaError_t prepare_linear_gemm_gelu();
cudaError_t prepare_linear_gemm_gelu_tanh();
cudaError_t prepare_linear_gemm_silu();
// CTA pairs that are resident at once.
int linear_pair_units(int sms);
// Once for a device; gives its error word.
cudaError_t prepare_linear_gemm(int32_t** error);
// The device's error word (CCE_DEVERR_*) of these kernels, taken and cleared behind `s`.
cudaError_t take_linear_error(int32_t* word, cudaStream_t s);
// A wait that runs out and sets `error` (cce_selftest_layers_wait_timeout).
cudaError_t launch_linear_wait_timeout(int32_t* error, uint64_t timeout_ns, cudaStream_t s);

// y = epilogue of the sums over the splits of a problem.
cudaError_t launch_linear_join(const LinProblem& p, bool gated, bool bf16, int sms, cudaStream_t s);

// Few rows: out[j][i] = epilogue(sum over k of w[i][k] x[j][k]), J <= LIN_FEW_ROWS.
struct LinFew {
  const void* w[2];
  int64_t w_pitch[2];
  const void* x;
  int64_t x_pitch;
  int I, J, K;
  LinEpilogue e;
};
// Beyond, a token more costs the GEMM nothing, and here a fourth tile of eight rows reads x again: 4,096 x 4,096 takes 9.8 us
// for 32 rows here, 10.4 for 33 there; 17 rows 8.3 here and 11.1 there.
constexpr int LIN_FEW_ROWS = 32;
cudaError_t launch_linear_few(const LinFew& a, bool gated, bool bf16, cudaStream_t s);

// The element-wise part of the backward pass: dz = dy f'(z) (gated: dgate = dy u
// f'(g) and dup = dy f(g)) in the operands' type, and the sums of dz over the rows.
struct LinGrad {
  const void* dy;
  int64_t dy_pitch;
  int dy_type;
  const void* z[2];
  int64_t z_pitch[2];
  int kept;  // z is CCE_KEPT16, else of the operands' type
  void* dz[2];  // may be null (sums alone)
  int64_t dz_pitch;
  float* part;  // [parts][N], may be null (no sums)
  int M, N, act;
};
constexpr int LIN_GRAD_PARTS = 256;
// How many parts of the sums there are, at most (whole vectors; fewer otherwise).
int linear_grad_parts(int64_t M, int64_t N);
// *parts: how many there are.
cudaError_t launch_linear_grad(const LinGrad& a, bool gated, bool bf16, cudaStream_t s, int* parts);
cudaError_t launch_linear_sum(const LinSum& a, cudaStream_t s);


// Rows of several matrices (include/cce_layers.h, cce_copy_rows); empty ones are left out.
struct LinCopies {
  cce_row_copy c[CCE_MAX_ROW_COPIES];
  int64_t first[CCE_MAX_ROW_COPIES];  // row of the launch at which each begins
  int64_t rows;
  int n;
};
cudaError_t launch_linear_copies(const LinCopies& a, int sms, cudaStream_t s);

}  // namespace cce

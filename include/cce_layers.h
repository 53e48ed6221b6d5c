/*
 * cce_layers.h -- C ABI of the layers in front of the classifier head: a matrix
 * product with bias, activation and residual in its epilogue, and the gated
 * product of a feed-forward block; forward and backward.
 *
 * Conventions are those of cce.h and cce_ops.h: plain device pointers and
 * sizes, the caller owns every buffer (workspaces included; the library
 * allocates no device memory), argument checks run before anything is launched
 * and return a cce_status, calls are asynchronous on `stream`, outputs are
 * overwritten and overlap no input.  Every result is deterministic: the order of
 * every sum is fixed by the sizes, types and alignments of the arguments, by which
 * results are asked for and by the device (a grad_x alone and one beside weight
 * gradients may sum in another order).
 *
 * Matrices
 * --------
 * Row-major with a pitch in elements.  The operands of a product (x, weights; z,
 * gate and up as well) are 16-bit, all CCE_BF16 or all CCE_F16: products of them
 * are exact in fp32 and are summed in fp32 on the tensor cores.  x and weights
 * start on 16 bytes and have pitches of a multiple of 8 elements, at least K, that
 * are below 2^31; what lies between a row's end and the next row's start is not
 * read into results and may hold anything (whole aligned words of 16 bytes that hold
 * an element are read).  Other matrices need the alignment of their element alone, and
 * pitches below 2^30.
 * Sizes: M >= 0 rows, < 2^31 - 512, N >= 1 outputs and K >= 1 inputs of a layer, both
 * < 2^30, any two of the three multiplied < 2^45.  Workspaces start on 256 bytes; where
 * a query gives 16, none is needed and it may be NULL.
 * M = 0 is fine: nothing is launched, or zero weight gradients are written.
 *
 * Activations
 * -----------
 * relu max(z, 0); gelu z Phi(z) with the normal distribution function, whose smaller
 * half is within (z^2 + 16) 2^-23 of its own value (below 2^-126 it may be 0); gelu_tanh
 * z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2; silu z / (1 + e^-z).  The
 * derivative of relu at 0 is 0.
 */
#ifndef CCE_LAYERS_GB300_H
#define CCE_LAYERS_GB300_H

#include "cce_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A type for what a forward pass keeps for its backward pass: 16 bits, a sign, 6 of
 * exponent (bias 31) and 9 of fraction, with subnormals, infinities and NaN as in IEEE's
 * types, to nearest.  Two bits of fraction more than bf16's between 2^-30 and 2^32;
 * values beyond become infinite, ones below 2^-40 zero.
 */
#define CCE_KEPT16 3

enum { CCE_ACT_NONE = 0, CCE_ACT_RELU = 1, CCE_ACT_GELU = 2, CCE_ACT_GELU_TANH = 3, CCE_ACT_SILU = 4 };

/* ABI version of this header (major * 100 + minor): 100. */
int cce_layers_abi_version(void);

/*
 * Linear layer, forward: z = x weight^T + bias, y = act(z) + residual.
 *
 *   x         [M, K] of `type`     weight    [N, K] of `type`
 *   bias      [N] of bias_type, any of the three types; NULL: 0
 *   residual  [M, N] of y_type, rows as of cce_ops.h ("Rows"); NULL: 0
 *   y         [M, N] of y_type: `type` or CCE_F32
 *   z         [M, N] of z_type, for the backward pass; NULL: not written.  z_type is
 *             `type`, or CCE_KEPT16 with CCE_BF16
 * Everything behind the product is fp32, with one rounding to y and one to z.
 */
cce_status cce_linear_forward(const void* x, int64_t x_pitch, const void* weight, int64_t w_pitch, int type,
                              const void* bias, int bias_type, const void* residual, int64_t r_inner, int64_t r_row_stride,
                              int64_t r_outer_stride, int act, int64_t M, int64_t N, int64_t K, void* y,
                              int64_t y_pitch, int y_type, void* z, int64_t z_pitch, int z_type, void* workspace,
                              size_t ws_bytes, void* stream);

/* Bytes of workspace (0 for invalid sizes; 16 where none is needed).  Pure host arithmetic; needs no GPU. */
size_t cce_linear_forward_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * Linear layer, backward.  With dz = grad_y act'(z), rounded to `type` for the
 * two products:
 *   grad_x = dz weight          [M, K] of `type`, dense
 *   grad_weight = dz^T x        [N, K] of `type`, dense
 *   grad_bias = sum of dz over the rows, in fp32 before that rounding
 *                               [N] of bias_type
 * Each may be NULL (not computed).  grad_y is [M, N] of y_type, `type` or
 * CCE_F32; z is the forward's, of z_type, or NULL with CCE_ACT_NONE.  The residual's
 * gradient is grad_y itself.
 */
cce_status cce_linear_backward(const void* grad_y, int64_t g_pitch, int y_type, const void* x, int64_t x_pitch,
                               const void* weight, int64_t w_pitch, int type, const void* z, int64_t z_pitch,
                               int z_type, int act, int64_t M, int64_t N, int64_t K, void* grad_x,
                               void* grad_weight, void* grad_bias, int bias_type, void* workspace, size_t ws_bytes,
                               void* stream);

/* Bytes of workspace, as above, for any call of these sizes; cce_layers_ex.h has what one call needs. */
size_t cce_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * Gated product, forward: gate = x gate_weight^T, up = x up_weight^T,
 * y = act(gate) up, of `type`; both weights [N, K].  gate and up [M, N] of one
 * pitch and of z_type (as above) are written for the backward pass unless both are NULL.
 */
cce_status cce_gated_linear_forward(const void* x, int64_t x_pitch, const void* gate_weight, int64_t gw_pitch,
                                    const void* up_weight, int64_t uw_pitch, int type, int act, int64_t M, int64_t N,
                                    int64_t K, void* y, int64_t y_pitch, void* gate, void* up, int64_t z_pitch,
                                    int z_type, void* workspace, size_t ws_bytes, void* stream);
size_t cce_gated_linear_forward_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * Gated product, backward.  With dgate = grad_y up act'(gate) and
 * dup = grad_y act(gate), both rounded to `type`:
 *   grad_x = dgate gate_weight + dup up_weight   [M, K], one fp32 sum
 *   grad_gate_weight = dgate^T x, grad_up_weight = dup^T x   [N, K]
 * Each may be NULL.  grad_y [M, N] of `type`, gate and up of z_type.
 */
cce_status cce_gated_linear_backward(const void* grad_y, int64_t g_pitch, const void* x, int64_t x_pitch,
                                     const void* gate_weight, int64_t gw_pitch, const void* up_weight,
                                     int64_t uw_pitch, int type, const void* gate, int64_t gate_pitch, const void* up,
                                     int64_t up_pitch, int z_type, int act, int64_t M, int64_t N, int64_t K,
                                     void* grad_x, void* grad_gate_weight, void* grad_up_weight, void* workspace, size_t ws_bytes,
                                     void* stream);
size_t cce_gated_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * Copies rows of up to CCE_MAX_ROW_COPIES matrices in one launch, for those whose
 * rows are not as the products take them: row n of the source starts (n / inner) *
 * outer_stride + (n % inner) * row_stride elements after src (strides >= 0, unit stride
 * inside a row, aligned words of 16 bytes that hold an element are read whole), row n of
 * the destination n * pitch elements after dst, on 16 bytes with a pitch of a multiple of
 * 16 bytes; what completes a row's last 16 bytes is written as zeros.  Elements of 2 or
 * 4 bytes, sources aligned to them.  Destinations overlap nothing.
 */
#define CCE_MAX_ROW_COPIES 8
typedef struct {
  const void* src;
  void* dst;
  int64_t inner, row_stride, outer_stride, pitch;
  int64_t rows, cols; /* either may be 0 */
  int32_t bytes;      /* of an element */
} cce_row_copy;

cce_status cce_copy_rows(const cce_row_copy* copies /* host */, int n, void* stream);

/*
 * *word (host) = the errors (CCE_DEVERR_*) that the products of this header met
 * on the current device since the last call, 0 without any; waits for `stream`.
 * Only a wait that ran out sets one: the results of its call are undefined.
 */
cce_status cce_layers_take_error(int32_t* word /* host */, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CCE_LAYERS_GB300_H */

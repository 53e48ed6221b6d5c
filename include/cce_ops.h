/*
 * cce_ops.h -- C ABI of the operators around the classifier head: the norm
 * that produces its hidden states E (layer norm, RMS norm; forward and
 * backward) and the global norm and clipping of the gradients that its
 * backward pass leaves.
 *
 * Conventions are those of cce.h: plain device pointers and sizes, the caller
 * owns every buffer (workspaces included; the library allocates no device
 * memory), argument checks run before anything is launched and return a
 * cce_status, calls are asynchronous on `stream`, outputs are overwritten.
 * Every result is deterministic: the order of every sum is fixed by the sizes,
 * types, strides and alignments of the arguments and by the device.
 *
 * Element types
 * -------------
 * CCE_F32, CCE_F16, CCE_BF16.  Arithmetic is fp32 throughout, with the sums of a
 * gradient norm as pairs of fp32 values; each output is rounded once, to nearest even.
 *
 * Rows
 * ----
 * A norm works on N rows of D elements, unit stride inside a row.  Inputs x
 * and grad_y may be strided views: row n starts (n / inner) * outer_stride +
 * (n % inner) * row_stride elements after the pointer (a plain matrix has
 * inner = N).  Strides are >= 0; rows of an input may coincide.  Of what lies
 * between the first and the last element of an input, aligned words of 16 bytes
 * that hold an element of a row may be read whole.  Outputs y and grad_x are
 * dense [N, D].  Outputs of a norm overlap no input.
 */
#ifndef CCE_OPS_GB300_H
#define CCE_OPS_GB300_H

#include "cce.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { CCE_F32 = 0, CCE_F16 = 1, CCE_BF16 = 2 } cce_type;

/* ABI version of this header (major * 100 + minor): 100. */
int cce_ops_abi_version(void);

/*
 * Layer norm, forward: per row
 *   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),
 *   y = (x - mean) * rstd * weight + bias.
 *
 *   x_type, y_type  equal, or x_type CCE_F32 with a 16-bit y_type (a 32-bit
 *                   residual stream normalised to 16-bit hidden states);
 *                   anything else returns CCE_ERR_ARG.
 *   weight, bias    [D] of p_type, each may be NULL (1 and 0).
 *   mean, rstd      [N] fp32 (written), each may be NULL; the backward needs
 *                   them.
 * N = 0 is fine (nothing is launched); D >= 1.  N, D < 2^31.  Pointers need the
 * alignment of their element.  Fastest are rows of a multiple of 16 bytes that
 * start on 16 bytes; next, matrices whose rows all start alike (any D, at least
 * 64, aligned pointers, pitches that differ from D by a multiple of 16 bytes of
 * x), then others of at least 64 columns.  A row whose squared deviations overflow fp32 gets rstd 0; one with
 * a NaN or an infinity, or whose sum overflows fp32, becomes NaN; the other rows keep their results.
 */
cce_status cce_layer_norm_forward(const void* x, int64_t x_inner, int64_t x_row_stride, int64_t x_outer_stride,
                                  int x_type, const void* weight, const void* bias, int p_type, int64_t N, int64_t D,
                                  float eps, void* y, int y_type, float* mean, float* rstd, void* stream);

/*
 * Layer norm, backward.  With z = (x - mean) * rstd and g = grad_y * weight:
 *   grad_x      = rstd * (g - sum(g) / D - z * sum(g z) / D)   [N, D], x_type
 *   grad_weight = sum over rows of grad_y * z                 [D], p_type
 *   grad_bias   = sum over rows of grad_y                     [D], p_type
 * Each of the three may be NULL (not computed).  mean and rstd are the
 * forward's.  The row sums are fp32: per-block partials in `workspace`, then
 * one fixed-order sum over the blocks.  N = 0 writes zero parameter gradients.
 */
cce_status cce_layer_norm_backward(const void* grad_y, int64_t g_inner, int64_t g_row_stride, int64_t g_outer_stride,
                                   int y_type, const void* x, int64_t x_inner, int64_t x_row_stride,
                                   int64_t x_outer_stride, int x_type, const void* weight, int p_type,
                                   const float* mean, const float* rstd, int64_t N, int64_t D, void* grad_x,
                                   void* grad_weight, void* grad_bias, void* workspace, size_t ws_bytes,
                                   void* stream);

/*
 * RMS norm, forward: y = x * rstd * (weight_offset + weight),
 * rstd = 1 / sqrt(sum x^2 / D + eps).  weight NULL: y = x * rstd.
 * weight_offset is 1 for models that store the weight minus one.
 */
cce_status cce_rms_norm_forward(const void* x, int64_t x_inner, int64_t x_row_stride, int64_t x_outer_stride,
                                int x_type, const void* weight, int p_type, float weight_offset, int64_t N, int64_t D,
                                float eps, void* y, int y_type, float* rstd, void* stream);

/* RMS norm, backward: with z = x * rstd and g = grad_y * (weight_offset +
 * weight), grad_x = rstd * (g - z * sum(g z) / D) and grad_weight = sum over
 * rows of grad_y * z.  grad_x and grad_weight may each be NULL. */
cce_status cce_rms_norm_backward(const void* grad_y, int64_t g_inner, int64_t g_row_stride, int64_t g_outer_stride,
                                 int y_type, const void* x, int64_t x_inner, int64_t x_row_stride,
                                 int64_t x_outer_stride, int x_type, const void* weight, int p_type,
                                 float weight_offset, const float* rstd, int64_t N, int64_t D, void* grad_x,
                                 void* grad_weight, void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace the backward of either norm needs (0 for invalid
 * sizes).  Pure host arithmetic; needs no GPU. */
size_t cce_norm_backward_workspace_bytes(int64_t N, int64_t D);

/*
 * Global gradient norm and clipping over any number of tensors.
 *
 * Tensors come as two host arrays, read during the call:
 *   dense    [n_dense][4] int64: {input pointer, output pointer, number of
 *            elements (0 is skipped), input type + 256 * output type}.  Input
 *            and output are contiguous blocks of memory in the same order.
 *   strided  n_strided descriptors of tensors whose elements are not one block.
 * Outputs are read by cce_clip_grads only.  An output is the input itself (in
 * place, same type and strides) or memory that overlaps no other input or
 * output: dense blocks that do overlap return CCE_ERR_ARG.
 */
typedef struct {
  const void* in;
  void* out;
  int32_t in_type, out_type;
  int64_t size[4];       /* dimensions, 1 where there are fewer; the last varies fastest */
  int64_t in_stride[4];  /* in elements, >= 0 */
  int64_t out_stride[4]; /* in elements, >= 0 */
} cce_strided;

#define CCE_NORM_INF 0
#define CCE_NORM_2 2

/*
 * *norm (fp32, device, written) = sqrt(sum x^2) (CCE_NORM_2) or max |x|
 * (CCE_NORM_INF) over all elements; 0 without any.  Where squares leave fp32's
 * range they are summed in fp64, so the norm is right wherever fp32 can hold it; an
 * infinity or NaN among the elements gives infinity or NaN.
 */
cce_status cce_grad_norm(const int64_t* dense /* host */, int64_t n_dense, const cce_strided* strided /* host */,
                         int64_t n_strided, int norm_type, float* norm, void* workspace, size_t ws_bytes,
                         void* stream);

/*
 * The norm as above, then output = input * min(1, max_norm / (norm + eps)),
 * rounded once to the output's type.  A factor of 1 leaves tensors that are
 * clipped in place untouched.  A NaN norm gives a factor of NaN.  An infinite
 * norm gives 0, or 1 if max_norm is infinite too; norm + eps = 0 gives 1.
 * max_norm >= 0 (infinity: never clip) and a finite eps >= 0, else CCE_ERR_ARG.
 */
cce_status cce_clip_grads(const int64_t* dense /* host */, int64_t n_dense, const cce_strided* strided /* host */,
                          int64_t n_strided, int norm_type, float max_norm, float eps, float* norm, void* workspace,
                          size_t ws_bytes, void* stream);

/* Bytes of workspace for that many tensors (0 for negative counts).  Pure
 * host arithmetic; needs no GPU. */
size_t cce_grad_norm_workspace_bytes(int64_t n_dense, int64_t n_strided);

#ifdef __cplusplus
}
#endif

#endif /* CCE_OPS_GB300_H */

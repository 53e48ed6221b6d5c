/*
 * cce_optim.h -- C ABI of the update that ends a training step of the head:
 * AdamW over any number of tensors, with states in 32 or in 8 bits.
 *
 * Conventions are those of cce.h and cce_ops.h.  No workspace is needed.  Every
 * result is deterministic.
 *
 * For each element, with g the gradient times min(1, max_norm / (norm + eps_norm)):
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   w = w (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32 (an eps below 2^-150 counts as 0, and 0 / 0 is NaN).  w is the fp32 master weight
 * where there is one, which is updated, and the parameter is w rounded once to its type.
 *
 * States in 8 bits
 * ----------------
 * Each tensor's values are in blocks of 256 in memory order, the last one shorter.
 * A block of m has an fp32 scale, its largest magnitude / 448, and e4m3 values that
 * stand for multiples of it; of v the square root is held the same way.  A new value a
 * (in multiples of the scale) is rounded at random: to a's upper neighbour in e4m3
 * with the distance from the lower one, in steps between them, as probability, so that
 * a moving average moves although one step's change is far below a rounding; m's
 * magnitude is what is rounded, and a positive root does not become 0 (the least
 * e4m3 value takes its place), so that no element is divided by eps alone.  A block
 * whose largest magnitude is below 2^-116 is held as zeros.  A NaN or infinity makes
 * its block's state NaN.
 *
 * The random numbers are those of (seed, t): with mix the finaliser of MurmurHash3
 * (x ^= x >> 16; x *= 0x85ebca6b; x ^= x >> 13; x *= 0xc2b2ae35; x ^= x >> 16),
 * key = mix(mix(seed) ^ (t mod 2^32)), and element e of the call's block b (counted
 * over its tensors in order) at p = 256 b + e, the word is
 * mix((p mod 2^32) ^ mix(key ^ (p >> 32))); its low 16 bits / 2^16 is m's number and
 * its high 16 bits / 2^16 v's, and a is rounded to floor(a / step + number) step.
 */
#ifndef CCE_OPTIM_GB300_H
#define CCE_OPTIM_GB300_H

#include "cce_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CCE_ADAMW_BLOCK 256

/* ABI version of this header (major * 100 + minor): 100. */
int cce_optim_abi_version(void);

/* One tensor: blocks of n elements in one order.  Empty ones (n = 0) are skipped. */
typedef struct {
  const void* grad;
  void* param;
  float* master;     /* NULL: the parameter itself is the weight */
  void* exp_avg;     /* m: fp32, or e4m3 */
  void* exp_avg_sq;  /* v: fp32; or its root: e4m3 */
  float* exp_avg_scale; /* 8 bits: ceil(n / 256) scales, else not read */
  float* rms_scale;
  int64_t n;
  int32_t grad_type, param_type;
  float weight_decay;
} cce_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps;
  int64_t step;           /* t >= 1 of this update; with step_ptr not read */
  const int64_t* step_ptr; /* device, may be NULL */
  const float* lr_ptr;    /* device, may be NULL: lr */
  const float* norm;      /* device, may be NULL: gradients are not clipped */
  float max_norm, eps_norm;
  uint32_t seed;
} cce_adamw_options;

/*
 * state_bits: 32 or 8.  tensors and options are host memory, read during the call.
 * CCE_ERR_ARG: betas outside of [0, 1), a negative or non-finite lr, eps, eps_norm or
 * weight_decay, a step below 1, a max_norm that is negative or NaN, or memory that is
 * written and overlaps another input or output.  A step_ptr that holds less than 1
 * counts as 1.  Pointers need the alignment of their element; on 16 bytes they are fastest.
 */
cce_status cce_adamw_step(const cce_adamw_tensor* tensors /* host */, int64_t n_tensors, int state_bits,
                          const cce_adamw_options* options /* host */, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CCE_OPTIM_GB300_H */

/*
 * cce_layers_ex.h -- more of the C ABI of the layers (cce_layers.h), whose conventions hold.
 */
#ifndef CCE_LAYERS_EX_GB300_H
#define CCE_LAYERS_EX_GB300_H

#include "cce_layers.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Tile plans are searched once for a combination of products and kept, some 1,000 of
 * them in a process: how many have been searched so far.  A call or query whose like was
 * made before adds none while they are kept.
 */
uint64_t cce_layers_plan_searches(void);

/*
 * Bytes of workspace of one backward call, which takes less than any (the queries of
 * cce_layers.h) where it computes less.  want: the results that are not NULL (DX grad_x, DW
 * grad_weight or grad_gate_weight, DW_UP grad_up_weight, DB grad_bias), and for a linear
 * layer DZ unless its products can read grad_y itself: act is CCE_ACT_NONE, y_type is `type`
 * and grad_y starts on 16 bytes at a pitch of a multiple of 8 elements (or neither DX nor DW
 * is wanted).  A call checks for no more than this.  0 for invalid sizes or flags.
 */
enum { CCE_WANT_DX = 1, CCE_WANT_DW = 2, CCE_WANT_DW_UP = 4, CCE_WANT_DB = 8, CCE_WANT_DZ = 16 };

size_t cce_linear_backward_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int want);
size_t cce_gated_linear_backward_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int want);

/*
 * Self-test of the failure path of the products' waits: one thread waits, as their roles do,
 * on a barrier that nothing arrives on; after timeout_us (1 .. 10^7) microseconds the wait
 * gives up and sets the device's error word, which cce_layers_take_error then gives
 * (CCE_DEVERR_TIMEOUT).  No fault, no hang: the context stays usable.
 */
cce_status cce_selftest_layers_wait_timeout(uint32_t timeout_us, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CCE_LAYERS_EX_GB300_H */

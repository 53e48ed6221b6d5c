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

#ifdef __cplusplus
}
#endif

#endif /* CCE_LAYERS_EX_GB300_H */

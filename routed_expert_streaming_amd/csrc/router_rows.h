// Router logits of many tokens in fp64, for the routers that choose from them.  (A header of
// its own: the fused kernels that finish the router of a few tokens read none of it.)
#pragma once
#include "common.h"

namespace moe {

// Logits [T][E] of more than 32 tokens on the fp64 matrix cores.
int router_logits_rows(const uint16_t *x, int T, int H, const float *w_router, const float *bias, int E, float *logits,
                       hipStream_t s);

}  // namespace moe

// Router logits on the bf16 matrix cores with a bound on their error.
#pragma once
#include "common.h"

namespace moe {

// logit[t,e] = sum of its parts (fp64), off by at most
//   split_error(columns of a part) * sqrt(sum of xn[.][t]) * sqrt(sum of wn[.][e])
struct RouterSplit {
    int parts, columns;            // of H: parts of `columns` columns, a multiple of 64
    size_t partial, xn, wn, total;  // byte offsets of one layer's fp32 [parts][T][E], [parts][T], [parts][E]; bytes
};
RouterSplit router_split_layout(int layers, int T, int E, int H);
int router_split(const uint16_t *x, int layers, int T, int H, const float *w_router, int E, const RouterSplit &sp,
                 void *workspace, hipStream_t s);

// Relative to sqrt(sum x^2) sqrt(sum w^2), which is at least the sum of the terms'
// magnitudes.  What v_mfma_f32_16x16x32_bf16 keeps (measured): of each 8 products (8
// neighbouring columns) the bits down to 2^-23 of the largest one's exponent; with the sums
// of eights and the addend rounded to fp32 it is off by at most (7 + 5) * 2^-24 of the
// magnitudes of its terms and its addend.  Per 64 columns the large plane takes two of them
// (12 * 2^-23 in all) and the small planes four on sums below 2^-7 of it; 16 leaves a
// third to spare.  Then one addition per 64 columns of the part (2^-24); 1.01 for the
// norms' own rounding.
__host__ __device__ inline float router_split_error(int columns) {
    return 1.01f * (16.0f + 0.5f * (float)(columns / 64 + 1)) * 0x1p-23f;
}

}  // namespace moe

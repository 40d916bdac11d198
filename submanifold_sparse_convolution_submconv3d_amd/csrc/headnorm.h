// Arguments of the heads' norm with rotation (headnorm.hip).
#pragma once

#include "rotary.h"

namespace sc {

struct HeadNormArgs {
    const void *x, *g;
    void *out;  // y, or dx
    int64_t x_row, x_head, g_row, g_head, out_row, out_head, pos_row, n;
    const int32_t *pos;
    const float *freqs;
    const void *w;
    float *rstd;     // [n, heads]
    float *partial;  // backward: [blocks][weight rows][dim]
    RotaryAxes ax;
    int heads, dim, pdtype, weight_rows, q_heads;
    int hb, rb;      // heads and rows a block works on at a time
    float eps;
};

size_t head_norm_bwd_workspace(int64_t n, int heads, int dim, int dtype, int weight_rows, int q_heads);
int head_norm(HeadNormArgs A, int dtype, int split, hipStream_t st);
int head_norm_backward(HeadNormArgs A, int dtype, int split, void *dw, hipStream_t st);

}  // namespace sc

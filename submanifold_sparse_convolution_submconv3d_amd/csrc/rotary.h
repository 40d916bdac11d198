// The angle of a pair of a head's elements at a position, shared by the rotation (rotary.hip)
// and the heads' norm with the rotation in the same pass (headnorm.hip).
#pragma once

#include "rowvec.h"

namespace sc {

struct RotaryAxes {
    int end[SUBMCONV_ROTARY_MAX_AXES];  // first pair past each axis' section
};

// cos and sin of position * freq.  The product and its reduction to one turn are in fp64
// (a position of 2^31 still leaves 1e-7 of a turn), the rest in fp32.
__device__ __forceinline__ void turn(int32_t position, float freq, bool inverse, float *c, float *s)
{
    const double rev = (double)position * (double)freq * 0.15915494309189533577;
    sincospif((float)(2.0 * (rev - rint(rev))), s, c);
    if (inverse) *s = -*s;
}

// The axis that pair p belongs to (the sections past the last axis end where it does).
__device__ __forceinline__ int rotary_axis(const RotaryAxes &ax, int p)
{
    int a = 0;
#pragma unroll
    for (int k = 0; k < SUBMCONV_ROTARY_MAX_AXES - 1; ++k) a += p >= ax.end[k];
    return a;
}

static inline RotaryAxes rotary_axes(const int32_t *sections, int axes)
{
    RotaryAxes ax;
    for (int a = 0, end = 0; a < SUBMCONV_ROTARY_MAX_AXES; ++a) ax.end[a] = end += a < axes ? sections[a] : 0;
    return ax;
}

}  // namespace sc

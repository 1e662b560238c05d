// The rotary embedding's arithmetic, one routine for every kernel that turns
// rows (kvattn_rope, kvattn_append_kv, kvattn_append_slots): pair i of a d-wide
// slice turned by pos * base^(-2i/d), angle and turn in double precision.  The
// products are written with their roundings, so that no kernel's compilation
// fuses them another way.
#pragma once

#include <math.h>

namespace kvattn {

// Radians that pair i of a d-wide slice turns per position.
__device__ __forceinline__ double rope_rate(int i, int d, double log2_base)
{
    return exp2(-2.0 * (double)i / (double)d * log2_base);
}

__device__ __forceinline__ void rope_angle(long long pos, double rate, double *s, double *c)
{
    sincos(__dmul_rn((double)pos, rate), s, c);
}

__device__ __forceinline__ void rope_turn(double x0, double x1, double s, double c, double *r0, double *r1)
{
    *r0 = __fma_rn(x0, c, -__dmul_rn(x1, s));
    *r1 = __fma_rn(x0, s, __dmul_rn(x1, c));
}

}  // namespace kvattn

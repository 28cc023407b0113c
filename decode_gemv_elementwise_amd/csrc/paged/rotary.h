// The turn of rotary positions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gemv {
namespace {

// (cos, sin) of pos * inv.  The angle is formed in 64 bits: a position of a million times
// a frequency near 1 has no correct fraction of a turn left in 32.  The 64-bit part is
// the product and the reduction to [-pi/4, pi/4], by pi / 2 in two parts (the double
// nearest, and what it lacks); there the Taylor series up to r^9 and r^10 are within
// 2e-9 (the next terms are (pi/4)^11 / 11! and (pi/4)^12 / 12!), well inside a 32-bit
// rounding.
__device__ __forceinline__ float2 turn_of(int32_t pos, float inv)
{
    const double a = (double)pos * (double)inv;
    const double k = rint(a * 0.63661977236758134308);
    double r = fma(-k, 1.57079632679489661923, a);
    r = fma(-k, 6.123233995736766e-17, r);
    const int quarter = (int)(k - 4.0 * floor(k * 0.25));
    const float x = (float)r, z = x * x;
    float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    s = fmaf(z, s, 8.3333333e-3f);
    s = fmaf(z, s, -1.6666667e-1f);
    s = fmaf(x * z, s, x);
    float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    c = fmaf(z, c, -1.3888889e-3f);
    c = fmaf(z, c, 4.1666667e-2f);
    c = fmaf(z, c, -0.5f);
    c = fmaf(z, c, 1.0f);
    const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
    return float2{quarter == 1 || quarter == 2 ? -cc : cc, quarter >= 2 ? -ss : ss};
}

} // namespace
} // namespace gemv

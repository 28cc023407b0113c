// The turn of rotary positions.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gemv {
namespace {

// An angle less whole quarters of a turn, and how many those are, 0..3.
struct Quarters {
    double rest; // in [-pi / 4, pi / 4]
    int count;
};

// The angle pos * inv is formed in 64 bits: a position of a million times a frequency near
// 1 has no correct fraction of a turn left in 32.  It is reduced by pi / 2 in two parts
// (the double nearest, and what it lacks).
__device__ __forceinline__ Quarters quarters_of(int32_t pos, float inv)
{
    const double a = (double)pos * (double)inv;
    const double k = rint(a * 0.63661977236758134308);
    double r = fma(-k, 1.57079632679489661923, a);
    r = fma(-k, 6.123233995736766e-17, r);
    return Quarters{r, (int)(k - 4.0 * floor(k * 0.25))};
}

// (cos, sin) of `quarter` quarters of a turn and the angle whose (cos, sin) are (c, s).
__device__ __forceinline__ float2 by_quarter(int quarter, float c, float s)
{
    const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
    return float2{quarter == 1 || quarter == 2 ? -cc : cc, quarter >= 2 ? -ss : ss};
}

// The Taylor series up to r^9 and r^10 of an angle of at most a quarter turn either way
// are within 2e-9 (the next terms are (pi/4)^11 / 11! and (pi/4)^12 / 12!), well inside a
// 32-bit rounding: sin x = x + x z sin_rest(z) and cos x = 1 - z / 2 + z^2 cos_rest(z),
// z = x^2.
__device__ __forceinline__ float sin_rest(float z)
{
    float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    s = fmaf(z, s, 8.3333333e-3f);
    return fmaf(z, s, -1.6666667e-1f);
}
__device__ __forceinline__ float cos_rest(float z)
{
    float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
    c = fmaf(z, c, -1.3888889e-3f);
    return fmaf(z, c, 4.1666667e-2f);
}

// (cos, sin) of pos * inv, within 7.1e-8 and 6.0e-8.
__device__ __forceinline__ float2 turn_of(int32_t pos, float inv)
{
    const Quarters a = quarters_of(pos, inv);
    const float x = (float)a.rest, z = x * x;
    const float s = fmaf(x * z, sin_rest(z), x);
    const float c = fmaf(z, fmaf(z, cos_rest(z), -0.5f), 1.0f);
    return by_quarter(a.count, c, s);
}

// The same within 3.5e-8 and 4.3e-8, against the 3.0e-8 of one rounding: with what x lacks
// of the angle and z of its square, and each sum's largest terms last.  For values that are
// rounded to few bits next, where each one that this moves over a border is off by a step.
__device__ __forceinline__ float2 turn_close(int32_t pos, float inv)
{
    const Quarters a = quarters_of(pos, inv);
    const float x = (float)a.rest, z = x * x, low = (float)(a.rest - (double)x);
    const float half = -0.5f * z, near = 1.0f + half;
    const float lack = fmaf(x, low, 0.5f * fmaf(x, x, -z)); // half of x's square beyond z
    const float c = near + (((1.0f - near) + half) + fmaf(z * z, cos_rest(z), -lack));
    const float s = x + fmaf(x * z, sin_rest(z), low * c);
    return by_quarter(a.count, c, s);
}

} // namespace
} // namespace gemv

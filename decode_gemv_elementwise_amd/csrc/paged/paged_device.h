// Device code shared by the paged operators: vector types, division by a page
// size, and sums over a wave and a workgroup.  Everything sits in an unnamed
// namespace, so each translation unit has its own copy.
#pragma once

#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "paged_internal.h"

namespace gemv {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;

__device__ __forceinline__ uint32_t div_by(FastDiv d, uint32_t n) { return (__umulhi(d.mul, n) + n) >> d.shift; }

// a + b, at most cap (a, b and cap below 2^31): associative, so a scan of it is
// the cut prefix sum.
__device__ __forceinline__ uint32_t add_cut(uint32_t a, uint32_t b, uint32_t cap)
{
    const uint32_t s = a + b;
    return s < cap ? s : cap;
}

// Exclusive prefix of v over a workgroup of WAVES waves; *total gets the whole
// sum.  `scratch` holds WAVES words and is free again after the caller's next
// barrier.
template <int WAVES, class T, class Add>
__device__ __forceinline__ T block_prefix(T v, T *scratch, T *total, Add add)
{
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    T s = v;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const T o = __shfl_up(s, d);
        if (lane >= d)
            s = add(o, s);
    }
    if (lane == kWave - 1)
        scratch[wave] = s;
    __syncthreads();
    T base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (w == wave)
            base = all;
        all = add(all, scratch[w]);
    }
    *total = all;
    const T before = __shfl_up(s, 1);
    return lane == 0 ? base : add(base, before);
}

} // namespace
} // namespace gemv

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

// Another lane's value by a DPP control; 0 where the lane has no source.
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}

// Exclusive prefix of v over a workgroup of WAVES waves; *total gets the whole
// sum (add(0, v) is v).  `scratch` holds WAVES words and is free again after the
// caller's next barrier.  Within a wave: shifts by 1, 2, 4 and 8 in rows of 16
// lanes, then each row's last lane to the rows after it.
template <int WAVES, class Add>
__device__ __forceinline__ uint32_t block_prefix(int thread, uint32_t v, uint32_t *scratch, uint32_t *total, Add add)
{
    const int lane = thread & (kWave - 1), wave = thread / kWave;
    uint32_t s = v;
    s = add(dpp<0x111, 0xf>(s), s);
    s = add(dpp<0x112, 0xf>(s), s);
    s = add(dpp<0x114, 0xf>(s), s);
    s = add(dpp<0x118, 0xf>(s), s);
    s = add(dpp<0x142, 0xa>(s), s);
    s = add(dpp<0x143, 0xc>(s), s);
    if (lane == kWave - 1)
        scratch[wave] = s;
    __syncthreads();
    uint32_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (w == wave)
            base = all;
        all = add(all, scratch[w]);
    }
    *total = all;
    return add(base, dpp<0x138, 0xf>(s));
}

} // namespace
} // namespace gemv

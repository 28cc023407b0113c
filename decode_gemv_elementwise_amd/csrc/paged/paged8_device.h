// Device code shared by the operators over a cache of 8-bit codes: scales, and codes
// widened to the types that are computed with.
#pragma once

#include "paged8_internal.h"
#include "paged_device.h"

namespace gemv {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

// The float that a scale's byte stands for (0 for byte 0, which is below what is kept).
__device__ __forceinline__ float scale_of(uint32_t byte)
{
    return __builtin_bit_cast(float, byte == 255 ? 0x7fc00000u : byte << 23);
}

// Two floats rounded to nearest into 16 bits.
template <bool BF> __device__ __forceinline__ uint32_t pack2(float x, float y)
{
    if constexpr (BF) {
        bf2_t r;
        r[0] = (__bf16)x;
        r[1] = (__bf16)y;
        return __builtin_bit_cast(uint32_t, r);
    } else {
        half2_t r;
        r[0] = (_Float16)x;
        r[1] = (_Float16)y;
        return __builtin_bit_cast(uint32_t, r);
    }
}

// Four codes, from a word's lowest byte up, times their scale, in 32 bits.
template <int CODE> __device__ __forceinline__ f32x4 floats4(uint32_t w, float scale)
{
    f32x4 x;
    // a word as it was loaded: where the compiler sees through a loop, it carries single
    // bytes from one turn to the next, a register each
    asm volatile("" : "+v"(w));
    if constexpr (CODE == GEMV_KV_E4M3) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        x = f32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = (float)((w ^ 0x80808080u) >> (8 * i) & 255) - 128.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] *= scale;
    return x;
}

// The same rounded to nearest into 16 bits, which changes nothing where they hold the
// product.
template <int CODE, bool BF> __device__ __forceinline__ u32x2 widen4(uint32_t w, float scale)
{
    if constexpr (CODE == GEMV_KV_E4M3 && BF) {
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))};
    } else if constexpr (CODE == GEMV_KV_E4M3) {
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true))};
    } else {
        const f32x4 x = floats4<CODE>(w, scale);
        return u32x2{pack2<BF>(x[0], x[1]), pack2<BF>(x[2], x[3])};
    }
}

template <int CODE, bool BF> __device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi, float scale)
{
    const u32x2 x = widen4<CODE, BF>(lo, scale), y = widen4<CODE, BF>(hi, scale);
    return u32x4{x[0], x[1], y[0], y[1]};
}

} // namespace
} // namespace gemv

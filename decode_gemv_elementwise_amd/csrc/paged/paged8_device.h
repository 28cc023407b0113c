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

// A word as it was loaded: where the compiler sees through a loop, it carries single
// bytes from one turn to the next, a register each.
__device__ __forceinline__ uint32_t whole_word(uint32_t w)
{
    asm volatile("" : "+v"(w));
    return w;
}

// Four codes, from a word's lowest byte up, in 32 bits.
template <int CODE> __device__ __forceinline__ f32x4 floats4(uint32_t w)
{
    if constexpr (CODE == GEMV_KV_E4M3) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
        return f32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
        f32x4 x;
        w = whole_word(w);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = (float)(int8_t)(w >> (8 * i));
        return x;
    }
}

// Four codes in 16 bits, which hold them exactly.  An int8 c goes to binary16 as the
// low bits of 1024 + (c + 128), less 1152: an instruction for two.
template <int CODE, bool BF> __device__ __forceinline__ u32x2 codes16(uint32_t w)
{
    if constexpr (CODE == GEMV_KV_E4M3 && BF) {
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
    } else if constexpr (CODE == GEMV_KV_E4M3) {
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))};
    } else if constexpr (BF) {
        const f32x4 x = floats4<CODE>(w);
        return u32x2{pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3])};
    } else {
        const half2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
        w = whole_word(w) ^ 0x80808080u;
        const half2_t lo = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u)) - off;
        const half2_t hi = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u)) - off;
        return u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
    }
}

// A scale as values of 16 bits are multiplied by it.  Binary16 holds the powers of two from
// 2^-24 to 2^15: there a whole number is multiplied by two, the first exactly.
template <int CODE, bool BF> struct Scale {
    float f;
    half2_t a, b;
    __device__ __forceinline__ explicit Scale(uint32_t byte) : f(scale_of(byte))
    {
        if constexpr (CODE == GEMV_KV_INT8 && !BF) {
            const int e = (int)byte - 127, e1 = min(max(e, -14), 9), e2 = min(max(e - e1, -25), 15);
            const _Float16 x = byte == 255 ? (_Float16)__builtin_nanf("") : (_Float16)ldexpf(1.0f, e1), y = (_Float16)ldexpf(1.0f, e2);
            a = half2_t{x, x};
            b = half2_t{y, y};
        }
    }
};

// Four codes times their scale, rounded to nearest into 16 bits, which changes nothing
// where they hold the product.
template <int CODE, bool BF> __device__ __forceinline__ u32x2 widen4(uint32_t w, const Scale<CODE, BF> &s)
{
    if constexpr (CODE == GEMV_KV_E4M3 && BF) {
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s.f, true))};
    } else if constexpr (CODE == GEMV_KV_E4M3) {
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s.f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s.f, true))};
    } else if constexpr (BF) {
        const f32x4 x = floats4<CODE>(w);
        return u32x2{pack2<true>(x[0] * s.f, x[1] * s.f), pack2<true>(x[2] * s.f, x[3] * s.f)};
    } else {
        const u32x2 c = codes16<CODE, false>(w);
        const uint32_t lo = c[0], hi = c[1];
        return u32x2{__builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, lo) * s.a * s.b),
                     __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, hi) * s.a * s.b)};
    }
}

template <int CODE, bool BF> __device__ __forceinline__ u32x4 widen8(uint32_t lo, uint32_t hi, const Scale<CODE, BF> &s)
{
    const u32x2 x = widen4<CODE, BF>(lo, s), y = widen4<CODE, BF>(hi, s);
    return u32x4{x[0], x[1], y[0], y[1]};
}

} // namespace
} // namespace gemv

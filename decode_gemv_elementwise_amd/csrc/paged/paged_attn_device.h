// What the two kinds of row tile of gemv_paged_attn share: arguments, element
// types, masks, the walk over a tile's keys and the exchange of parts.
#pragma once

#include <type_traits>

#include "paged_device.h"

namespace gemv {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr float kNegInf = -__builtin_inff();
// A weight 2^(s - m) of binary16 is carried 2^14 times its size (the sums l and
// over v alike, so it cancels): its smallest step, 2^-24, would otherwise lose
// the many small weights of a long row beside one large one.  It is added to s - m:
// folded into m it is lost, or grows to 16 and past binary16, where m is so large
// that a step of 32 bits is 2 or more.
constexpr float kF16Lift = 14.0f;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct AttnArgs {
    const uint16_t *q, *k, *v;
    int64_t q_ts, q_hs, o_ts, o_hs;
    uint32_t k_stride[3], v_stride[3]; // below 2^31
    const int32_t *table, *query_start, *kv_len;
    int64_t table_stride;
    void *out;
    int32_t *counters;
    float *parts;
    int64_t part_room;           // floats that the workspace has for parts
    int32_t width, requests, tokens, heads, group, num_pages, window, sinks, unit_log2, tile_cost;
    int64_t reach;               // keys that a table row can hold
    float scale_log2;            // |scale| log2(e); its sign is in q_flip
    uint32_t q_keep, q_flip;     // q's words are (x & q_keep) ^ q_flip: scale 0 takes q as 0
    FastDiv page, per_group;
};

// This thread's index, as far as the compiler knows another one at each call: what
// is worked out from it stays where it is used.  Carried over from share to share
// (of both kinds of tile) it would be spilled.
__device__ __forceinline__ int thread_here()
{
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// True for every thread if it is for one.  flags: a word a wave, free again after
// the caller's next barrier.
__device__ __forceinline__ bool any_thread(int thread, bool x, uint32_t *flags)
{
    const uint32_t mine = __any(x);
    if ((thread & (kWave - 1)) == 0)
        flags[thread / kWave] = mine;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        all |= flags[w];
    return uniform(all);
}

template <bool BF> __device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

template <bool BF> __device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
{
    if constexpr (BF)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// Eight floats rounded to nearest into 16 bits.
template <bool BF> __device__ __forceinline__ u32x4 round8(const float *p)
{
    typedef typename std::conditional<BF, bf16x8, f16x8>::type T8;
    typedef typename std::conditional<BF, __bf16, _Float16>::type T;
    T8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = (T)p[i];
    return __builtin_bit_cast(u32x4, r);
}

// Two floats rounded to nearest into 16 bits.
template <bool BF> __device__ __forceinline__ uint32_t round2(const float *p)
{
    typedef typename std::conditional<BF, __bf16, _Float16>::type T;
    typedef T t2 __attribute__((ext_vector_type(2)));
    t2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r[i] = (T)p[i];
    return __builtin_bit_cast(uint32_t, r);
}

// Two floats from 0 up as two pieces of 16 bits each, for a result of 32: the first
// piece is returned, p gets the rest.  The first lies below p, so that the rest is
// above 0 and an infinity of v times either is that infinity; a piece of 0, which
// rounding to nearest leaves of a weight of 1, would make it NaN.  Together they are
// within 2^-16 (bf16) and 2^-21 (binary16) of p.
template <bool BF> __device__ __forceinline__ uint32_t split2(float *p)
{
    if constexpr (BF) {
        const uint32_t a = __builtin_elementwise_sub_sat(__builtin_bit_cast(uint32_t, p[0]), 1u);
        const uint32_t b = __builtin_elementwise_sub_sat(__builtin_bit_cast(uint32_t, p[1]), 1u);
        p[0] -= __builtin_bit_cast(float, a & 0xffff0000u);
        p[1] -= __builtin_bit_cast(float, b & 0xffff0000u);
        return __builtin_amdgcn_perm(b, a, 0x07060302u);
    } else {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const u16x2 r = __builtin_elementwise_sub_sat(
            __builtin_bit_cast(u16x2, __builtin_amdgcn_cvt_pkrtz(p[0], p[1])), u16x2{1, 1});
        const f16x2 f = __builtin_bit_cast(f16x2, r);
        p[0] -= (float)f[0];
        p[1] -= (float)f[1];
        return __builtin_bit_cast(uint32_t, r);
    }
}

template <bool BF> __device__ __forceinline__ float as_float(uint16_t x)
{
    if constexpr (BF)
        return __builtin_bit_cast(float, (uint32_t)x << 16);
    else
        return (float)__builtin_bit_cast(_Float16, x);
}

// Bits 15 and 31 are set where that half is an infinity or NaN: adding one to a
// full exponent carries into the sign's place, and the sign is masked off.
template <bool BF> __device__ __forceinline__ uint32_t not_finite(uint32_t x)
{
    constexpr uint32_t e = BF ? 0x7f807f80u : 0x7c007c00u, one = BF ? 0x00800080u : 0x04000400u;
    return ((x & e) + one) & 0x80008000u;
}

// Four results, rounded to the output's type, to 4-aligned places of a row.
template <bool BF, bool F32OUT> __device__ __forceinline__ void store4(void *out, int64_t at, f32x4 x)
{
    if constexpr (F32OUT) {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(out) + at) = x;
    } else {
        typedef typename std::conditional<BF, __bf16, _Float16>::type T;
        typedef T t4 __attribute__((ext_vector_type(4)));
        t4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = (T)x[e];
        *reinterpret_cast<t4 *>(static_cast<T *>(out) + at) = y;
    }
}

struct Request {
    int q0, n, kv;
};

__device__ __forceinline__ Request request_of(const AttnArgs &a, int r)
{
    const int q0 = min(max(a.query_start[r], 0), a.tokens), q1 = min(max(a.query_start[r + 1], q0), a.tokens);
    return Request{q0, q1 - q0, max(a.kv_len[r], 0)};
}

// The keys of one row tile in blocks of B: blocks [0, first) hold the first
// tokens that stay visible, then blocks from `skip` on.
struct Walk {
    int first, skip, count;
    __device__ __forceinline__ int block(int i) const { return i < first ? i : i - first + skip; }
};

template <int B> __device__ __forceinline__ Walk walk_of(const AttnArgs &a, int p_lo, int p_hi)
{
    const int64_t end = min((int64_t)p_hi + 1, a.reach);
    if (end <= 0)
        return Walk{0, 0, 0};
    const int all = (int)((end + B - 1) / B);
    if (a.window == 0)
        return Walk{0, 0, all};
    const int first = (int)((min((int64_t)a.sinks, end) + B - 1) / B);
    const int64_t lo = max((int64_t)0, (int64_t)p_lo - a.window + 1);
    const int skip = max((int)min(lo / B, (int64_t)all), first);
    return Walk{first, skip, first + max(0, all - skip)};
}

__device__ __forceinline__ bool sees(const AttnArgs &a, int p_row, int j)
{
    return j <= p_row && (a.window == 0 || j > p_row - a.window || j < a.sinks);
}

// Every row from p_lo to p_hi sees every key of [j0, j0 + n).
__device__ __forceinline__ bool sees_all(const AttnArgs &a, int p_lo, int p_hi, int j0, int n)
{
    return j0 + n - 1 <= p_lo && (a.window == 0 || j0 > p_hi - a.window || j0 + n <= a.sinks);
}

// A scalar the compiler may not read again from the arguments: in a loop over keys
// that would be waited for at every block.
template <class T> __device__ __forceinline__ T kept(T x)
{
    asm volatile("" : "+s"(x));
    return x;
}

// What finds a key in the cache.
struct Paging {
    FastDiv page;
    uint32_t width, pages, k0, k1, v0, v1; // strides of page and of token in page

    // The page id of key j as the table has it, -1 past the table's end.
    __device__ __forceinline__ int raw(const int32_t *table, int j) const
    {
        const uint32_t at = div_by(page, j);
        return at < width ? table[at] : -1;
    }
    // -1 for what is no page.
    __device__ __forceinline__ int checked(int id) const { return (uint32_t)id < pages ? id : -1; }
    // Element offset of key j in page id (a key without a page reads page 0, and
    // what is read is dropped).
    template <bool V> __device__ __forceinline__ uint64_t offset(int id, int j) const
    {
        const uint32_t in = j - div_by(page, j) * page.d;
        return (uint64_t)(uint32_t)max(id, 0) * (V ? v0 : k0) + (uint64_t)in * (V ? v1 : k1);
    }
};

__device__ __forceinline__ Paging paging_of(const AttnArgs &a)
{
    return Paging{{kept(a.page.mul), kept(a.page.shift), kept(a.page.d)}, kept((uint32_t)a.width), kept((uint32_t)a.num_pages),
                  kept(a.k_stride[0]), kept(a.k_stride[1]), kept(a.v_stride[0]), kept(a.v_stride[1])};
}

// A workgroup's share of the keys of one row tile: of np workgroups it is the
// me-th, and takes from b to b + len of the nb blocks that the plan counts.  With
// np > 1 its sums go to part `mine`, and the last of the np to arrive joins all.
struct Share {
    int b, len, nb;
    int np, me;
    int first; // workgroup that has the tile's first block; index of its counter
    int stride; // floats from one part's place to the next
    __device__ __forceinline__ int from(int count) const { return (int)((int64_t)count * b / nb); }
    __device__ __forceinline__ int to(int count) const { return (int)((int64_t)count * (b + len) / nb); }
    // A workgroup ends at most one tile that others began and begins at most one
    // that others end: two places each.
    __device__ __forceinline__ int part(int i) const { return (2 * (first + i) + (i == 0)) * stride; }
};

// Parts go to memory and come from it past the caches that other units do not
// share (scope bit 16: the device), so no cache has to be written back or emptied
// for them: that costs a release and an acquire several us each.
struct Parts {
    __amdgpu_buffer_rsrc_t all;
    __device__ explicit Parts(const AttnArgs &a)
        : all(__builtin_amdgcn_make_buffer_rsrc(a.parts, 0, (int)min(a.part_room * 4, (int64_t)INT_MAX), 0x00020000))
    {
    }
    // at: floats from the first part's start, below 2^28
    __device__ __forceinline__ void put4(int at, f32x4 x) const
    {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), all, at * 4, 0, 16);
    }
    __device__ __forceinline__ void put(int at, float x) const
    {
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), all, at * 4, 0, 16);
    }
    __device__ __forceinline__ f32x4 get4(int at) const
    {
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(all, at * 4, 0, 16));
    }
    __device__ __forceinline__ float get(int at) const
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(all, at * 4, 0, 16));
    }
};

// Counts this workgroup's part as written; true for the one that came last.
// Every wave waits until its stores are where all units see them, then the
// barrier, then thread 0 counts.
__device__ __forceinline__ bool last_part(const AttnArgs &a, const Share &sh, int thread, int *lds)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (thread == 0) {
        const int before = __hip_atomic_fetch_add(a.counters + sh.first, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *lds = before == sh.np - 1;
        if (before == sh.np - 1) // ready for the next call
            __hip_atomic_store(a.counters + sh.first, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *lds;
}

} // namespace
} // namespace gemv

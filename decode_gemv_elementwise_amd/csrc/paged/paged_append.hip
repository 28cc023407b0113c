// Rotary positions and the write into the paged cache (gemv_paged_append).
//
// Memory-bound: every value of q, k and v is read once and written once, so
// the kernel is one pass with 16-byte accesses: 8192 tokens of 32 + 2 x 8 heads of
// 128 in 40.6 us, 4.96 TB/s read and written, where a large copy reaches 4.87 (42.6
// with a loop over tokens around it).  A workgroup takes one token
// (or, for few tokens, a share of one token's heads): its first threads form
// the cosines and sines of that token's rot / 2 angles, once for all heads,
// while the workgroup's first rows are on their way from memory.
//
// The angle is formed in 64 bits: a position of a million times a frequency
// near 1 has no correct fraction of a turn left in 32 bits.  The 64-bit part is
// the product and the reduction to [-pi/4, pi/4]; there the sine's and cosine's
// Taylor series up to r^9 and r^10 are within 2e-9 (the next terms are
// (pi/4)^11 / 11! and (pi/4)^12 / 12!), well inside a 32-bit rounding.
#include "paged_device.h"

namespace gemv {
namespace {

constexpr int kThreads = 256, kTokensX = 65536;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct AppendArgs {
    const void *src[3]; // q, k, v
    int64_t src_stride[3];
    const int32_t *positions, *axis, *slots;
    const float *inv_freq;
    void *q_out, *k, *v;
    int64_t k_stride[3], v_stride[3];
    int32_t tokens, axes, q_heads, heads, dim, half, pairs; // half = rot / 2
    int64_t num_slots;
    FastDiv page, turn_items, v_items; // items per head of q and k, and of v
    int32_t total;                     // items of one token
};

template <class T> struct Vec8;
template <> struct Vec8<_Float16> {
    typedef f16x8 type;
};
template <> struct Vec8<__bf16> {
    typedef bf16x8 type;
};

// (cos, sin) of pos * inv.  pi / 2 in two parts: the first is the double
// nearest, the second what it lacks.
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

// Eight values of a row from element e on, as floats.
template <class S> __device__ __forceinline__ void load8(const S *p, float *v)
{
    if constexpr (sizeof(S) == 4) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
        const typename Vec8<S>::type a = *reinterpret_cast<const typename Vec8<S>::type *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (float)a[i];
    }
}

template <class D> __device__ __forceinline__ void store8(D *p, const float *v)
{
    typename Vec8<D>::type a;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a[i] = (D)v[i];
    *reinterpret_cast<typename Vec8<D>::type *>(p) = a;
}

// One token's cosines and sines, by the workgroup's first threads.
__device__ __forceinline__ void fill_turns(const AppendArgs &a, int t, float2 *turns)
{
    for (int i = threadIdx.x; i < a.half; i += kThreads) {
        const int ax = a.axis ? a.axis[i] : 0;
        turns[i] = (unsigned)ax < (unsigned)a.axes ? turn_of(a.positions[(int64_t)ax * a.tokens + t], a.inv_freq[i])
                                                   : float2{1.0f, 0.0f};
    }
}

// Where a head's row of this token goes, or null (k and v of a token without a
// place).
template <class D>
__device__ __forceinline__ D *row_out(const AppendArgs &a, int t, int which, int head, int slot)
{
    if (which == 0)
        return static_cast<D *>(a.q_out) + ((int64_t)t * a.q_heads + head) * a.dim;
    if (slot < 0 || slot >= a.num_slots)
        return nullptr;
    const int64_t *s = which == 1 ? a.k_stride : a.v_stride;
    const uint32_t id = div_by(a.page, slot);
    return static_cast<D *>(which == 1 ? a.k : a.v) + id * s[0] + (slot - id * a.page.d) * s[1] + head * s[2];
}

// Splits a token's item into tensor, head and place within the head.
__device__ __forceinline__ void item_of(const AppendArgs &a, int item, int *which, int *head, int *at)
{
    const int turned = (a.q_heads + a.heads) * (int)a.turn_items.d;
    if (item < turned) {
        const int h = div_by(a.turn_items, item);
        *at = item - h * a.turn_items.d;
        *which = h < a.q_heads ? 0 : 1;
        *head = h < a.q_heads ? h : h - a.q_heads;
    } else {
        item -= turned;
        *head = div_by(a.v_items, item);
        *at = item - *head * a.v_items.d;
        *which = 2;
    }
}

// A workgroup's token: a grid's x counts its threads in 32 bits, so past 2^16
// tokens z goes on.
__device__ __forceinline__ int token_here() { return blockIdx.z * kTokensX + blockIdx.x; }

// The wide path.  An item is 8 neighbouring values, or for halves 8 values of
// the first half together with their 8 partners: rot is a multiple of 16 for
// halves (8 for pairs), so no vector straddles the halves or the end of rot.
template <class S, class D, bool PAIRS>
__global__ __launch_bounds__(kThreads) void paged_append_kernel(AppendArgs a)
{
    extern __shared__ float2 turns[];
    const int t = token_here();
    if (t >= a.tokens)
        return;
    const int slot = a.slots[t];
    bool filled = false;
    for (int item = blockIdx.y * kThreads + threadIdx.x;; item += gridDim.y * kThreads) {
        // the first rows are asked for before the angles are formed
        int which = 0, head = 0, at = 0, lo = 0, hi = 0;
        float u[8], w[8];
        const bool live = item < a.total;
        bool turn = false, two = false;
        if (live) {
            item_of(a, item, &which, &head, &at);
            if (PAIRS) {
                lo = 8 * at;
                turn = which < 2 && lo < 2 * a.half;
            } else {
                two = which < 2 && 8 * at < a.half;
                turn = two;
                lo = which < 2 && !two ? a.half + 8 * at : 8 * at;
                hi = lo + a.half;
            }
            const S *row = static_cast<const S *>(a.src[which]) + (int64_t)t * a.src_stride[which] + head * a.dim;
            load8(row + lo, u);
            if (two)
                load8(row + hi, w);
        }
        if (!filled) {
            fill_turns(a, t, turns);
            __syncthreads();
            filled = true;
        }
        if (live) {
            if (turn) {
#pragma unroll
                for (int i = 0; i < (PAIRS ? 4 : 8); ++i) {
                    float &x = PAIRS ? u[2 * i] : u[i], &y = PAIRS ? u[2 * i + 1] : w[i];
                    const float2 cs = turns[PAIRS ? lo / 2 + i : lo + i];
                    const float nx = fmaf(x, cs.x, -(y * cs.y)), ny = fmaf(y, cs.x, x * cs.y);
                    x = nx;
                    y = ny;
                }
            }
            if (D *out = row_out<D>(a, t, which, head, slot)) {
                store8(out + lo, u);
                if (two)
                    store8(out + hi, w);
            }
        }
        if (item - (int)threadIdx.x + (int)(gridDim.y * kThreads) >= a.total)
            break;
    }
}

// Any alignment and any even rot: an item is one value, or a pair's two.
template <class S, class D>
__global__ __launch_bounds__(kThreads) void paged_append_generic_kernel(AppendArgs a)
{
    extern __shared__ float2 turns[];
    const int t = token_here();
    if (t >= a.tokens)
        return;
    const int slot = a.slots[t];
    fill_turns(a, t, turns);
    __syncthreads();
    for (int item = blockIdx.y * kThreads + threadIdx.x; item < a.total; item += gridDim.y * kThreads) {
        int which, head, at;
        item_of(a, item, &which, &head, &at);
        const S *row = static_cast<const S *>(a.src[which]) + (int64_t)t * a.src_stride[which] + head * a.dim;
        D *out = row_out<D>(a, t, which, head, slot);
        if (!out)
            continue;
        if (which < 2 && at < a.half) {
            const int lo = a.pairs ? 2 * at : at, hi = a.pairs ? lo + 1 : lo + a.half;
            const float x = (float)row[lo], y = (float)row[hi];
            const float2 cs = turns[at];
            out[lo] = (D)fmaf(x, cs.x, -(y * cs.y));
            out[hi] = (D)fmaf(y, cs.x, x * cs.y);
        } else {
            const int e = which < 2 ? a.half + at : at;
            out[e] = (D)(float)row[e];
        }
    }
}

template <class S, class D> const void *kernel_of(bool wide, bool pairs)
{
    if (!wide)
        return reinterpret_cast<const void *>(&paged_append_generic_kernel<S, D>);
    return pairs ? reinterpret_cast<const void *>(&paged_append_kernel<S, D, true>)
                 : reinterpret_cast<const void *>(&paged_append_kernel<S, D, false>);
}

template <class S> const void *kernel_of(int type, bool wide, bool pairs)
{
    return type == GEMV_W_F16 ? kernel_of<S, _Float16>(wide, pairs) : kernel_of<S, __bf16>(wide, pairs);
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged_append(const void *q, const void *k, const void *v, int src_type, int64_t tokens,
                                 int64_t q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                 const int32_t *positions, int64_t axes, const int32_t *axis, const float *inv_freq,
                                 int64_t rot, int style, const int32_t *slots, void *q_out,
                                 const gemv_kv_cache *cache, void *hip_stream)
{
    const int st = gemv::validate_append(q, k, v, src_type, tokens, q_heads, q_stride, k_stride, v_stride, positions,
                                         axes, axis, inv_freq, rot, style, slots, q_out, cache);
    if (st != GEMV_OK)
        return st;
    if (tokens == 0)
        return gemv::finish_launch((int)hipSuccess);
    gemv::AppendArgs a{};
    a.src[0] = q, a.src[1] = k, a.src[2] = v;
    a.src_stride[0] = q_stride, a.src_stride[1] = k_stride, a.src_stride[2] = v_stride;
    a.positions = positions, a.axis = axis, a.slots = slots, a.inv_freq = inv_freq;
    a.q_out = q_out, a.k = cache->k, a.v = cache->v;
    for (int d = 0; d < 3; ++d)
        a.k_stride[d] = cache->k_stride[d], a.v_stride[d] = cache->v_stride[d];
    a.tokens = (int)tokens, a.axes = (int)axes, a.q_heads = (int)q_heads, a.heads = cache->heads, a.dim = cache->dim;
    a.half = (int)(rot / 2), a.pairs = style == GEMV_ROPE_PAIRS;
    a.num_slots = cache->num_pages * cache->page_size;
    a.page = gemv::fast_div(cache->page_size);

    // wide: 16-byte vectors of whole rows.  The cache and q_out always allow
    // them (checked strides and alignment); the rows of q, k and v and rot may not.
    const int64_t size = src_type == GEMV_W_F32 ? 4 : 2;
    bool wide = rot % (a.pairs ? 8 : 16) == 0;
    for (int i = 0; i < 3; ++i)
        wide = wide && reinterpret_cast<uintptr_t>(a.src[i]) % 16 == 0 && a.src_stride[i] * size % 16 == 0;
    const int step = wide ? 8 : 1;
    a.turn_items = gemv::fast_div((wide && a.pairs ? a.dim : a.dim - a.half) / step);
    a.v_items = gemv::fast_div(a.dim / step);
    a.total = (a.q_heads + a.heads) * (int)a.turn_items.d + a.heads * (int)a.v_items.d;

    // One workgroup per token fills the card from a few hundred tokens on; below
    // that a token's items are spread over enough workgroups to give every
    // thread one.
    const int64_t most = (a.total + gemv::kThreads - 1) / gemv::kThreads;
    int64_t parts = (512 + tokens - 1) / tokens;
    parts = parts < most ? parts : most;
    const void *fn = src_type == GEMV_W_F32   ? gemv::kernel_of<float>(cache->type, wide, a.pairs)
                     : src_type == GEMV_W_F16 ? gemv::kernel_of<_Float16>(cache->type, wide, a.pairs)
                                              : gemv::kernel_of<__bf16>(cache->type, wide, a.pairs);
    void *args[] = {&a};
    const int64_t x = tokens < gemv::kTokensX ? tokens : gemv::kTokensX;
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)x, (unsigned)parts, (unsigned)((tokens + x - 1) / x)),
                                         dim3(gemv::kThreads), args, (size_t)a.half * sizeof(float2),
                                         static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}

// Tokens of a paged cache of 8-bit codes in 16 or 32 bits (gemv_paged8_read).
//
// Memory-bound: a byte read and two or four written a value.  A thread makes 16 bytes of
// a row of the result from 4 or 8 neighbouring codes of one head, and asks for four such
// pieces before it uses one.  65536 tokens of 8 heads of 128 to bf16 take 84 us, 4.80 TB/s:
// a copy's rate; 100 tokens 3.7 us, a launch.
#include "paged8_device.h"

namespace gemv {
namespace {

constexpr int kThreads = 256, kAhead = 4; // pieces of a thread, all asked for before any is used

struct Read8Args {
    const uint8_t *codes[2], *scales[2]; // k, v
    const int32_t *slots;
    void *out[2];
    int64_t c_stride[2][3], s_stride[2][3], out_stride[2];
    int32_t tokens, first; // first: the tensor of the grid's first y (1: v alone)
    int32_t per_z;         // tokens of one step of the grid's z
    int32_t num_slots;
    FastDiv page, block, row, head; // pieces of a token, pieces of a head
};

template <int CODE, int TYPE> __global__ __launch_bounds__(kThreads) void paged8_read_kernel(Read8Args a)
{
    constexpr int E = TYPE == GEMV_W_F32 ? 4 : 8; // codes of a piece
    const int v = a.first + blockIdx.y;
    const uint8_t *const codes = v ? a.codes[1] : a.codes[0], *const scales = v ? a.scales[1] : a.scales[0];
    const int64_t *const c = v ? a.c_stride[1] : a.c_stride[0], *const s = v ? a.s_stride[1] : a.s_stride[0];
    const int64_t t0 = (int64_t)blockIdx.z * a.per_z;
    const int n = (int)min((int64_t)a.per_z, a.tokens - t0);
    uint32_t w[kAhead][E / 4];
    int byte[kAhead]; // the scale's, -1 where there is no token, -2 past the end
    int64_t to[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const uint32_t at = (blockIdx.x * kAhead + i) * kThreads + threadIdx.x;
        const uint32_t t = div_by(a.row, at), piece = at - t * a.row.d;
        byte[i] = -2;
        if (t >= (uint32_t)n)
            continue;
        const uint32_t head = div_by(a.head, piece), e = (piece - head * a.head.d) * E;
        const int slot = a.slots[t0 + t];
        to[i] = (t0 + t) * (v ? a.out_stride[1] : a.out_stride[0]) + (int64_t)piece * E;
        byte[i] = -1;
        if (slot < 0 || slot >= a.num_slots)
            continue;
        const uint32_t id = div_by(a.page, slot), in = slot - id * a.page.d;
        const uint8_t *from = codes + id * c[0] + in * c[1] + head * c[2] + e;
        if constexpr (E == 4) {
            w[i][0] = *reinterpret_cast<const uint32_t *>(from);
        } else {
            const u32x2 x = *reinterpret_cast<const u32x2 *>(from);
            w[i][0] = x[0];
            w[i][1] = x[1];
        }
        byte[i] = scales[id * s[0] + div_by(a.block, in) * s[1] + head * s[2]];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        if (byte[i] == -2)
            continue;
        u32x4 y = {0, 0, 0, 0};
        if (byte[i] >= 0) {
            const Scale<CODE, TYPE == GEMV_W_BF16> scale(byte[i]);
            if constexpr (TYPE == GEMV_W_F32)
                y = __builtin_bit_cast(u32x4, floats4<CODE>(w[i][0]) * scale.f);
            else
                y = widen8<CODE, TYPE == GEMV_W_BF16>(w[i][0], w[i][E / 4 - 1], scale);
        }
        char *const out = static_cast<char *>(v ? a.out[1] : a.out[0]);
        *reinterpret_cast<u32x4 *>(out + to[i] * (16 / E)) = y;
    }
}

template <int CODE> const void *kernel_of(int type)
{
    return type == GEMV_W_F32   ? reinterpret_cast<const void *>(&paged8_read_kernel<CODE, GEMV_W_F32>)
           : type == GEMV_W_F16 ? reinterpret_cast<const void *>(&paged8_read_kernel<CODE, GEMV_W_F16>)
                                : reinterpret_cast<const void *>(&paged8_read_kernel<CODE, GEMV_W_BF16>);
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged8_read(const gemv_kv_cache8 *cache, const int32_t *slots, int64_t tokens, void *k_out, void *v_out,
                                int out_type, int64_t k_out_stride, int64_t v_out_stride, void *hip_stream)
{
    const int st = gemv::validate_read8(cache, slots, tokens, k_out, v_out, out_type, k_out_stride, v_out_stride);
    if (st != GEMV_OK)
        return st;
    if (tokens == 0)
        return gemv::finish_launch((int)hipSuccess);
    gemv::Read8Args a{};
    a.codes[0] = static_cast<const uint8_t *>(cache->k), a.codes[1] = static_cast<const uint8_t *>(cache->v);
    a.scales[0] = cache->k_scale, a.scales[1] = cache->v_scale;
    a.slots = slots, a.out[0] = k_out, a.out[1] = v_out;
    for (int d = 0; d < 3; ++d) {
        a.c_stride[0][d] = cache->k_stride[d], a.c_stride[1][d] = cache->v_stride[d];
        a.s_stride[0][d] = cache->ks_stride[d], a.s_stride[1][d] = cache->vs_stride[d];
    }
    a.out_stride[0] = k_out_stride, a.out_stride[1] = v_out_stride;
    a.tokens = (int)tokens, a.first = k_out ? 0 : 1;
    a.num_slots = (int)(cache->num_pages * cache->page_size);
    a.page = gemv::fast_div(cache->page_size), a.block = gemv::fast_div(cache->block);
    const int64_t piece = out_type == GEMV_W_F32 ? 4 : 8, row = cache->heads * (cache->dim / piece);
    a.row = gemv::fast_div(row), a.head = gemv::fast_div(cache->dim / piece);
    // pieces of one z are counted in 31 bits, those past the last token among them
    const int64_t span = gemv::kAhead * gemv::kThreads, most = ((1ll << 30) - span) / row;
    const int64_t per = tokens < most ? tokens : most, z = (tokens + per - 1) / per;
    a.per_z = (int)per;
    const void *fn = cache->code == GEMV_KV_INT8 ? gemv::kernel_of<GEMV_KV_INT8>(out_type)
                                                 : gemv::kernel_of<GEMV_KV_E4M3>(out_type);
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)((per * row + span - 1) / span), k_out && v_out ? 2 : 1, (unsigned)z),
                                         dim3(gemv::kThreads), args, 0, static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}

// Block tables and slot maps from request lengths (gemv_paged_slots).
//
// Everything is two prefix sums over the requests (tokens before a request,
// pages taken before it) and an expansion of both.  The requests are few and
// the expansion is wide, so every workgroup forms the sums itself, 1024
// requests at a time in LDS, and expands a 256-wide slice of the tokens, of the
// pages taken and of the requests: no workgroup waits for another, and one
// launch does it all.  A token's page comes from the free list directly where
// it is new, never from a table entry that another workgroup writes.
//
// Latency-bound: two dependent reads from memory and the scan between them.  3.7 us
// on the GPU for 64 requests with a token each, 5.4 for 1024 with 62000 together.
#include "paged_device.h"

namespace gemv {
namespace {

constexpr int kThreads = 256, kPer = 4, kChunk = kThreads * kPer;

struct SlotsArgs {
    const int32_t *cached, *fresh, *free_pages;
    int32_t *table, *query_start, *kv_len, *token_request, *positions, *slots, *used;
    int32_t requests, num_free, table_width, tokens;
    int64_t table_stride;
    FastDiv page;
};

// The last entry of a[0..n) that is <= v; a[0] <= v.
__device__ __forceinline__ int last_at_most(const uint32_t *a, int n, uint32_t v)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a[mid] <= v)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ uint32_t pages_of(FastDiv page, uint32_t tokens)
{
    return tokens == 0 ? 0 : div_by(page, tokens - 1) + 1;
}

__global__ __launch_bounds__(kThreads) void paged_slots_kernel(SlotsArgs a)
{
    __shared__ uint32_t start[kChunk], taken[kChunk], held[kChunk], scratch[2 * (kThreads / kWave)];
    const uint32_t tokens = a.tokens;
    const uint32_t mine = blockIdx.x * kThreads + threadIdx.x; // token, page taken and request of this thread
    uint32_t tbase = 0, pbase = 0;                             // tokens and pages before the chunk
    auto cut = [tokens](uint32_t x, uint32_t y) { return add_cut(x, y, tokens); };
    auto sum = [](uint32_t x, uint32_t y) { return x + y; };

    for (int r0 = 0; r0 < a.requests; r0 += kChunk) {
        uint32_t c[kPer], f[kPer], run = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = r0 + threadIdx.x * kPer + i;
            const int32_t cr = r < a.requests ? a.cached[r] : 0, fr = r < a.requests ? a.fresh[r] : 0;
            c[i] = cr > 0 ? cr : 0;
            f[i] = fr > 0 ? min((uint32_t)fr, (uint32_t)INT_MAX - c[i]) : 0;
            run = add_cut(run, min(f[i], tokens), tokens);
        }
        uint32_t all, at = block_prefix<kThreads / kWave>(threadIdx.x, run, scratch, &all, cut);
        at = add_cut(tbase, at, tokens);
        const uint32_t tend = add_cut(tbase, all, tokens);
        uint32_t need = 0, p[kPer], s[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t next = add_cut(at, min(f[i], tokens), tokens);
            s[i] = at;
            f[i] = next - at; // cut at the capacity
            at = next;
            p[i] = need;
            need += pages_of(a.page, c[i] + f[i]) - pages_of(a.page, c[i]);
        }
        const uint32_t pat = pbase + block_prefix<kThreads / kWave>(threadIdx.x, need, scratch + kThreads / kWave, &all, sum);
        const uint32_t pend = pbase + all;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = threadIdx.x * kPer + i;
            start[k] = s[i];
            taken[k] = pat + p[i];
            held[k] = c[i];
        }
        __syncthreads();
        const int n = min(kChunk, a.requests - r0);

        if (mine >= (uint32_t)r0 && mine < (uint32_t)(r0 + n)) {
            const int k = mine - r0;
            a.query_start[mine] = start[k];
            a.kv_len[mine] = held[k] + ((k + 1 < n ? start[k + 1] : tend) - start[k]);
        }
        if (mine >= pbase && mine < pend) {
            const int k = last_at_most(taken, n, mine);
            const uint32_t j = pages_of(a.page, held[k]) + (mine - taken[k]);
            if (j < (uint32_t)a.table_width)
                a.table[(r0 + k) * a.table_stride + j] = mine < (uint32_t)a.num_free ? a.free_pages[mine] : -1;
        }
        if (mine >= tbase && mine < tend) {
            const int k = last_at_most(start, n, mine);
            const uint32_t pos = held[k] + (mine - start[k]), j = div_by(a.page, pos), old = pages_of(a.page, held[k]);
            int32_t id = -1;
            if (j < (uint32_t)a.table_width) {
                if (j < old)
                    id = a.table[(r0 + k) * a.table_stride + j];
                else if (taken[k] + (j - old) < (uint32_t)a.num_free)
                    id = a.free_pages[taken[k] + (j - old)];
            }
            const int64_t slot = id < 0 ? -1 : (int64_t)id * a.page.d + (pos - j * a.page.d);
            a.token_request[mine] = r0 + k;
            a.positions[mine] = pos;
            a.slots[mine] = slot > INT_MAX ? -1 : (int32_t)slot;
        }
        tbase = tend;
        pbase = pend;
        __syncthreads();
    }
    if (mine >= tbase && mine < tokens) {
        a.token_request[mine] = -1;
        a.positions[mine] = 0;
        a.slots[mine] = -1;
    }
    if (mine == 0) {
        a.query_start[a.requests] = tbase;
        a.used[0] = min(pbase, (uint32_t)INT_MAX);
    }
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged_slots(const int32_t *cached, const int32_t *fresh, int64_t requests,
                                const int32_t *free_pages, int64_t num_free, int64_t page_size, int32_t *block_table,
                                int64_t table_width, int64_t table_stride, int64_t tokens, int32_t *query_start,
                                int32_t *kv_len, int32_t *token_request, int32_t *positions, int32_t *slots,
                                int32_t *used, void *hip_stream)
{
    const int st = gemv::validate_slots(cached, fresh, requests, free_pages, num_free, page_size, block_table,
                                        table_width, table_stride, tokens, query_start, kv_len, token_request,
                                        positions, slots, used);
    if (st != GEMV_OK)
        return st;
    gemv::SlotsArgs a{cached,         fresh,             free_pages,           block_table,      query_start,
                      kv_len,         token_request,     positions,            slots,            used,
                      (int)requests,  (int)num_free,     (int)table_width,     (int)tokens,      table_stride,
                      gemv::fast_div(page_size)};
    // a request takes at most ceil(fresh / page) pages: tokens / page + requests in all
    int64_t wide = tokens / page_size + requests;
    wide = wide > tokens ? wide : tokens;
    wide = wide > requests ? wide : requests;
    void *args[] = {&a};
    const hipError_t e =
        hipLaunchKernel(reinterpret_cast<const void *>(&gemv::paged_slots_kernel),
                        dim3((unsigned)((wide + gemv::kThreads - 1) / gemv::kThreads)), dim3(gemv::kThreads), args, 0,
                        static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}

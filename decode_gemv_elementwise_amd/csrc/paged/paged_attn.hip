// Attention of a request's new tokens over its paged cache (gemv_paged_attn).
//
// Mathematics: with s_j = scale q.k_j, the softmax is formed in one pass over
// the keys with the running maximum m and sum l of the rows, in powers of two
// (scale log2(e) folded into s): a block of keys with maximum b moves m to
// m' = max(m, b), scales l and the sums over v by 2^(m - m'), and adds
// 2^(s_j - m') v_j.  Parts of a row's keys join by the same rule.
//
// The rows of a request are its (token, query head) pairs, those that share a
// key/value head together.  Up to 16 of them are a tile of few rows
// (paged_attn_few.h), bound by the cache's bytes; more are cut into tiles of 128
// (64 for the widest heads)
// (paged_attn_many.h), bound by the matrix cores.
//
// The host does not know the lengths, so every workgroup works the plan out from
// them: the blocks of keys of all tiles form one line (request, head, tile,
// block), from a prefix sum over the requests, and workgroup w takes the w-th
// equal share of it, whatever tiles that cuts (but for slivers).  A tile whose keys are cut leaves
// its parts in the workspace; the workgroup that counts the last of them joins
// them in order, so the result does not depend on which came last.
#include <cfloat>
#include <cmath>

#include "paged_attn_few.h"
#include "paged_attn_many.h"

namespace gemv {
namespace {

// In blocks of 32 keys: what a workgroup takes at least, and how near a tile's edge
// a share's end moves to it.  Starting on a tile, and joining its parts, cost about
// as much as the blocks of `edge`.  One token over 4099 keys of 128-wide heads:
// shares of 8 at least 15.6 us, of 16 17.4; with edges of 2 17.6.  A mixed step of
// 16 requests, 64 wide: edges of 24 37.5 us, of 8 44.8; shares of 32 and edges of 40
// 40.4.  Drafts of up to 35 rows, 256 wide: shares of 8 33.5 us, of 4 37.0, of 12
// 42.9; requests of 3 keys there 12 us, with edges of 4, which cut their tiles, 24.
constexpr uint32_t least_share(int dim) { return dim == 64 ? 16 : 8; }
constexpr uint32_t few_edge(int dim) { return least_share(dim); }
constexpr uint32_t many_edge(int dim) { return dim == 64 ? 24 : dim == 128 ? 12 : 8; }
constexpr uint32_t kMostCost = INT_MAX;

// Up to 16 rows go by the waves' own way: one token over 4099 keys 15.6 us against
// 26.9 by a tile of many rows, over 131072 keys 105 against 125, 64 single tokens
// over up to 16384 keys 413 against 425.
__device__ __forceinline__ bool is_few(const AttnArgs &a, const Request &q) { return (int64_t)q.n * a.group <= kFewRows; }

template <int D> __device__ __forceinline__ uint32_t tiles_of(const AttnArgs &a, const Request &q)
{
    const uint32_t rows = (uint32_t)q.n * a.group; // below 2^31, as all rows together
    return is_few(a, q) ? rows != 0 : (rows + many_rows(D) - 1) / many_rows(D);
}

// What the plan counts for a row tile of the request: its blocks of 32 keys, the
// most that one tile visits (in units of 2^unit_log2 blocks, which is 1 unless
// the line would be longer than 2^31), and tile_cost for starting on it: many
// short tiles then spread over the card (21 requests of 16 keys and 8 heads each
// took 62 us where ten workgroups shared them).
template <int D> __device__ __forceinline__ uint32_t cost_of(const AttnArgs &a, const Request &q)
{
    uint32_t keys = (uint32_t)min((int64_t)q.kv, a.reach);
    if (a.window != 0) {
        const uint32_t some = (uint32_t)a.window + min(q.n, many_rows(D)) + 4 * kFewBlock; // below 2^32
        keys = min(keys, min((uint32_t)a.sinks, keys) + min(some, keys));
    }
    return ((keys + kFewBlock - 1) / kFewBlock >> a.unit_log2) + a.tile_cost;
}

// The kernel's arguments, read again from here on: the two kinds of tile need
// many of them, and holding all through both would cost registers in both.
__device__ __forceinline__ const AttnArgs &arguments()
{
    auto p = (const __attribute__((address_space(4))) AttnArgs *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttnArgs *)p;
}

template <bool BF, int D, bool F32OUT, int PAGES>
__global__ __launch_bounds__(kThreads, 2) void paged_attn_kernel(AttnArgs)
{
    const AttnArgs &a = arguments();
    // a buffer holds a block's rows, or a wave's sums of few rows
    constexpr int kBlockBytes = many_block(D) * 2 * D, kFewBytes = kFewRows * (D + 4) * 4;
    constexpr int kBuffer = kBlockBytes > kFewBytes ? kBlockBytes : kFewBytes;
    static_assert(many_part(D) <= attn_part_floats(D) && few_part(D) <= attn_part_floats(D), "the workspace's parts");
    __shared__ __align__(16) char ka[kBuffer];
    __shared__ __align__(16) char va[kBuffer];
    __shared__ __align__(16) char kb[kBuffer];
    __shared__ __align__(16) char vb[kBuffer];
    __shared__ uint32_t before[kThreads], scratch[kWaves], flags[kWaves];
    __shared__ Request requests[kThreads];

    // The line's length: requests that do not share rows stay below kMostCost (the
    // host chose the unit so); where query_start falls again, sums stop there.
    const auto sum = [](uint32_t x, uint32_t y) { return min(x + y, kMostCost); };
    const bool once = a.requests <= kThreads;
    uint32_t total = 0;
    bool many = false;
    if (!once) {
        uint32_t cost = 0;
        for (int r = threadIdx.x; r < a.requests; r += kThreads) {
            const Request q = request_of(a, r);
            cost = sum(cost, min((uint64_t)tiles_of<D>(a, q) * a.heads * cost_of<D>(a, q), (uint64_t)kMostCost));
            many = many || !is_few(a, q);
        }
        block_prefix<kWaves>(threadIdx.x, cost, scratch, &total, sum);
        total = uniform(total);
        many = any_thread(threadIdx.x, many, flags);
    }

    // this workgroup's share [x, x1): every group has `each` places, the first `more` one in addition
    uint32_t base = 0, x = 0, x1 = 0, each = 0, more = 0;
    int stride = 0;
    uint32_t edge = 0;
    // Neighbouring shares go to one of the 8 dies, which share an L2 cache; and where
    // a compute unit holds two workgroups, w and w + 256 in order of launch, the
    // second half of a die's shares goes backwards: later tiles of a chunk see more
    // keys, so a unit gets a long and a short one.
    uint32_t w = blockIdx.x;
    if (gridDim.x == kAttnGroups) {
        constexpr uint32_t per = kAttnGroups / 8;
        const uint32_t i = w / 8;
        w = w % 8 * per + (i < per / 2 ? i : per + per / 2 - 1 - i);
    }
    for (int r0 = 0; r0 < a.requests; r0 += kThreads) {
        const int thread = thread_here(), r = r0 + thread;
        Request q{0, 0, 0};
        if (r < a.requests)
            q = request_of(a, r);
        uint32_t here;
        before[thread] = block_prefix<kWaves>(
            thread, (uint32_t)min((uint64_t)tiles_of<D>(a, q) * a.heads * cost_of<D>(a, q), (uint64_t)kMostCost), scratch, &here, sum);
        requests[thread] = q;
        here = uniform(here);
        const bool any = any_thread(thread, !is_few(a, q), flags);
        if (r0 == 0) {
            if (once) {
                total = here;
                many = any;
            }
            const uint32_t groups = uniform(min(gridDim.x, (total + least_share(D) - 1) / least_share(D)));
            if (w >= groups || total == kMostCost)
                return;
            each = uniform(total / groups);
            more = total - each * groups;
            x = w * each + min(w, more);
            x1 = x + each + (w < more);
            // a tile is cut only if the parts have room: two for each workgroup, below 2^28 floats in all
            stride = many ? many_part(D) : few_part(D);
            edge = a.part_room < 2 * (int64_t)groups * stride ? kMostCost / 2 : many ? many_edge(D) : few_edge(D);
        }
        while (x < x1 && x < base + here) {
            int lo = 0, hi = min(kThreads, a.requests - r0);
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (before[mid] <= x - base)
                    lo = mid;
                else
                    hi = mid;
            }
            lo = uniform(lo);
            const Request q = {(int)uniform(requests[lo].q0), (int)uniform(requests[lo].n), (int)uniform(requests[lo].kv)};
            const uint32_t y = x - base - uniform(before[lo]), nb = uniform(cost_of<D>(a, q)), tiles = uniform(tiles_of<D>(a, q));
            const uint32_t unit = uniform(y / nb), start = x - (y - unit * nb); // of the tile
            // both ends of the share, as places of this tile; one near an edge of it moves there
            const auto moved = [&](uint32_t b) {
                return b >= nb ? nb : b < edge && b <= nb - b ? 0 : nb - b < edge && nb - b < b ? nb : b;
            };
            const uint32_t b0 = moved(x - start), b1 = moved(x1 - start);
            x = start + nb;
            if (b0 >= b1)
                continue;
            Share sh{(int)b0, (int)(b1 - b0), (int)nb, 1, 0, 0, stride};
            if (sh.len < (int)nb) {
                const auto group_of = [&](uint32_t place) {
                    const uint32_t longer = more * (each + 1);
                    return uniform(place < longer ? place / (each + 1) : more + (place - longer) / each);
                };
                sh.first = group_of(start + edge - 1);
                sh.np = group_of(start + nb - edge) - sh.first + 1;
                sh.me = w - sh.first;
            }
            const int head = uniform(unit / tiles), tile = unit - head * tiles;
            if (is_few(a, q))
                run_few<BF, D, F32OUT, PAGES>(arguments(), q, r0 + lo, head, sh, reinterpret_cast<float *>(ka),
                                              reinterpret_cast<float *>(va), reinterpret_cast<float *>(kb),
                                              reinterpret_cast<float *>(vb));
            else
                run_many<BF, D, F32OUT, PAGES>(arguments(), q, r0 + lo, tile, head, sh, ka, va, kb, vb);
        }
        if (x >= x1)
            return;
        base += here;
        __syncthreads();
    }
}

template <bool BF, int D, bool F32OUT> const void *kernel_of(int pages)
{
    return pages == 16  ? reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, F32OUT, 16>)
           : pages == 8 ? reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, F32OUT, 8>)
                        : reinterpret_cast<const void *>(&paged_attn_kernel<BF, D, F32OUT, 0>);
}

template <int D> const void *kernel_of(int type, bool f32out, int pages)
{
    if (type == GEMV_W_BF16)
        return f32out ? kernel_of<true, D, true>(pages) : kernel_of<true, D, false>(pages);
    return f32out ? kernel_of<false, D, true>(pages) : kernel_of<false, D, false>(pages);
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                               const gemv_kv_cache *cache, const int32_t *block_table, int64_t table_width,
                               int64_t table_stride, const int32_t *query_start, const int32_t *kv_len,
                               int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                               int64_t sinks, void *out, int out_type, int64_t out_token_stride,
                               int64_t out_head_stride, void *workspace, int64_t workspace_bytes, void *hip_stream)
{
    const int st = gemv::validate_attn(q, q_token_stride, q_head_stride, cache, block_table, table_width, table_stride,
                                       query_start, kv_len, requests, tokens, q_heads, scale, window, sinks, out,
                                       out_type, out_token_stride, out_head_stride, workspace, workspace_bytes);
    if (st != GEMV_OK)
        return st;
    if (tokens == 0)
        return gemv::finish_launch((int)hipSuccess);
    gemv::AttnArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(cache->k);
    a.v = static_cast<const uint16_t *>(cache->v);
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = out_token_stride, a.o_hs = out_head_stride;
    for (int d = 0; d < 3; ++d)
        a.k_stride[d] = (uint32_t)cache->k_stride[d], a.v_stride[d] = (uint32_t)cache->v_stride[d];
    a.table = block_table, a.query_start = query_start, a.kv_len = kv_len, a.table_stride = table_stride;
    a.out = out;
    const int64_t room = (workspace_bytes - gemv::kAttnCounters * 4) / 4;
    a.counters = static_cast<int32_t *>(workspace);
    a.parts = reinterpret_cast<float *>(a.counters + gemv::kAttnCounters);
    a.part_room = room < 0 ? 0 : room;
    a.width = (int)table_width, a.requests = (int)requests, a.tokens = (int)tokens, a.heads = cache->heads;
    a.group = (int)(q_heads / cache->heads), a.num_pages = (int)cache->num_pages;
    a.window = (int)window, a.sinks = window > 0 ? (int)sinks : 0;
    a.reach = table_width * cache->page_size; // a block's last key stays below 2^31
    a.reach = a.reach < INT_MAX - 63 ? a.reach : INT_MAX - 63;
    const float s = std::fabs(scale) * 1.44269504088896340736f;
    a.scale_log2 = s == 0.0f ? 1.0f : std::fmin(s, FLT_MAX);
    a.q_keep = s == 0.0f ? 0u : ~0u;
    a.q_flip = scale < 0.0f && s != 0.0f ? 0x80008000u : 0u;
    a.page = gemv::fast_div(cache->page_size), a.per_group = gemv::fast_div(a.group);

    const bool f32out = out_type == GEMV_W_F32;
    // Keys from a multiple of 16 (or 8) on that lie in one page are found once for all;
    // copies of 16 take 32-bit offsets within a run.  2048 new tokens over 8192 keys,
    // pages of 16: 273 us so, 340 by runs of 8 or key by key; one token over 131072
    // keys 105 us by runs of 16 or 8, 111 key by key.
    const bool near = a.k_stride[1] < (1u << 27) && a.v_stride[1] < (1u << 27);
    const int pages = cache->page_size % 16 == 0 && near ? 16 : cache->page_size % 8 == 0 ? 8 : 0;
    const void *fn = cache->dim == 64    ? gemv::kernel_of<64>(cache->type, f32out, pages)
                     : cache->dim == 128 ? gemv::kernel_of<128>(cache->type, f32out, pages)
                                         : gemv::kernel_of<256>(cache->type, f32out, pages);
    // no more workgroups than shares can be: row tiles times the blocks that the
    // table's width allows
    const int64_t blocks = (a.reach + gemv::kFewBlock - 1) / gemv::kFewBlock;
    int64_t tiles = tokens * a.group / gemv::kFewRows + (requests < tokens ? requests : tokens);
    tiles = (tiles < tokens * a.group ? tiles : tokens * a.group) * a.heads; // at most tokens * q_heads, below 2^31
    const int64_t cap = (INT_MAX - 1) / tiles; // of a tile's cost
    const int64_t start = gemv::least_share(cache->dim);
    a.tile_cost = (int)(start <= cap / 2 ? start : cap > 1 ? cap / 2 : 1);
    while (a.tile_cost + (blocks >> a.unit_log2) > cap)
        ++a.unit_log2;
    const int64_t most = gemv::kAttnGroups;
    const int64_t shares = (blocks + a.tile_cost) / gemv::least_share(128) + 1;
    const int grid = (int)(tiles >= most || shares >= most || tiles * shares >= most ? most : tiles * shares);
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid), dim3(gemv::kThreads), args, 0,
                                         static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}

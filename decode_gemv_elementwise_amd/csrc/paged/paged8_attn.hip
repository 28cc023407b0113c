// gemv_paged8_attn: what the host works out for the attention over a cache of 8-bit codes.
#include <cfloat>
#include <cmath>

#include "paged8_attn_device.h"

namespace gemv {
namespace {

// Which kind of row tile a call takes: one for the whole call, since the host knows the
// counts of tokens and requests and no lengths.  Few rows where there are no more tokens
// than requests, whatever the group, and where a request has two tiles of 16 rows or less on
// average.  us by few rows and by many, 8 requests over 4096 keys, heads of 128 in e4m3:
//     group 4, 8 key/value heads   20 rows 27 27   32 28 27   36 49 33   64 41 34   128 61 45
//     group 7, 4                   21      20 27   35 30 31   49 28 32   70 37 39   133 52 35
//     group 16, 2                  32      21 24   48 23 31   64 21 32   128 27 48
//     group 64, 1                  128     20 44
// so with few key/value heads it gives up early, and late with single tokens of such groups
// (64 query heads over one, 16384 keys: 1 request 27 43, 8 35 54, 64 130 94).  The mean is
// wrong where rows are spread unevenly: 512 single tokens over 100 keys and a chunk of 2000
// go by few rows (256 162; over 512 keys 280 259), and so does a chunk of 2000 among 500
// requests without tokens (213 74); 8 single tokens in a captured call of 512 go by many
// (over 4096 keys 24 27, over 16384 66 82).  It is right for 64 over 16384 keys with a chunk
// of 256 (584 693) or 2048 (1984 1107), and for 128 over 2048 with a chunk of 256 (136 177).
bool takes_many(int64_t tokens, int64_t requests, int64_t group)
{
    return tokens > requests && tokens * group > 2 * kAttnRows * requests;
}

} // namespace
} // namespace gemv

extern "C" int gemv_paged8_attn(const void *q, int q_type, int64_t q_token_stride, int64_t q_head_stride,
                                const gemv_kv_cache8 *cache, const int32_t *block_table, int64_t table_width,
                                int64_t table_stride, const int32_t *query_start, const int32_t *kv_len,
                                int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                                int64_t sinks, void *out, int out_type, int64_t out_token_stride,
                                int64_t out_head_stride, void *workspace, int64_t workspace_bytes, void *hip_stream)
{
    const int st = gemv::validate_attn8(q, q_type, q_token_stride, q_head_stride, cache, block_table, table_width,
                                        table_stride, query_start, kv_len, requests, tokens, q_heads, scale, window,
                                        sinks, out, out_type, out_token_stride, out_head_stride, workspace,
                                        workspace_bytes);
    if (st != GEMV_OK)
        return st;
    if (tokens == 0)
        return gemv::finish_launch((int)hipSuccess);
    gemv::Attn8Args a{};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(cache->k);
    a.v = static_cast<const uint16_t *>(cache->v);
    a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
    a.q_ts = q_token_stride, a.q_hs = q_head_stride, a.o_ts = out_token_stride, a.o_hs = out_head_stride;
    for (int d = 0; d < 3; ++d) {
        a.k_stride[d] = (uint32_t)cache->k_stride[d], a.v_stride[d] = (uint32_t)cache->v_stride[d];
        a.ks_stride[d] = (uint32_t)cache->ks_stride[d], a.vs_stride[d] = (uint32_t)cache->vs_stride[d];
    }
    a.table = block_table, a.query_start = query_start, a.kv_len = kv_len, a.table_stride = table_stride;
    a.out = out;
    const int64_t room = (workspace_bytes - gemv::kAttnCounters * 4) / 4;
    a.counters = static_cast<int32_t *>(workspace);
    a.parts = reinterpret_cast<float *>(a.counters + gemv::kAttnCounters);
    a.part_room = room < 0 ? 0 : room;
    a.width = (int)table_width, a.requests = (int)requests, a.tokens = (int)tokens, a.heads = cache->heads;
    a.group = (int)(q_heads / cache->heads), a.num_pages = (int)cache->num_pages;
    a.window = (int)window, a.sinks = window > 0 ? (int)sinks : 0;
    a.reach = table_width * cache->page_size; // a round's last key stays below 2^31
    a.reach = a.reach < INT_MAX - 63 ? a.reach : INT_MAX - 63;
    const float s = std::fabs(scale) * 1.44269504088896340736f;
    a.scale_log2 = s == 0.0f ? 1.0f : std::fmin(s, FLT_MAX);
    a.q_keep = s == 0.0f ? 0u : ~0u;
    a.q_flip = scale < 0.0f && s != 0.0f ? 0x80008000u : 0u;
    a.page = gemv::fast_div(cache->page_size), a.block = gemv::fast_div(cache->block);
    a.per_group = gemv::fast_div(a.group);

    const bool many = gemv::takes_many(tokens, requests, a.group);
    // where neighbouring keys lie: found once for all of a run, or key by key
    // 16 rows' offsets, and those of their scales, stay below 2^31
    const bool near = a.k_stride[1] < (1u << 27) && a.v_stride[1] < (1u << 27) && a.ks_stride[1] < (1u << 27) &&
                      a.vs_stride[1] < (1u << 27);
    const bool runs = !many ? cache->block % 8 == 0
                            : near && cache->page_size % 16 == 0 && (cache->block % 16 == 0 || 16 % cache->block == 0);
    const bool f32out = out_type == GEMV_W_F32, bf = q_type == GEMV_W_BF16;
    const void *fn = cache->dim == 64    ? gemv::paged8_attn_kernel_64(cache->code, bf, f32out, runs, many)
                     : cache->dim == 128 ? gemv::paged8_attn_kernel_128(cache->code, bf, f32out, runs, many)
                                         : gemv::paged8_attn_kernel_256(cache->code, bf, f32out, runs, many);
    // Where a token's heads lie one after the other in memory, rows of 128 bytes and less
    // are read by tiles of several of them: 64 single tokens over up to 16384 keys each,
    // 8 heads of 128 in e4m3, 203 us by four heads, 214 by two and 226 by one (196 where a
    // page's rows of one head lie together); of 64 130, 133 and 180; of 256 280, 266 and 265.
    // Tiles enough have to be left, or one is cut into so many parts that joining them takes
    // longest: one request of 131072 keys 106 us by four heads, 72 by one.
    const bool apart = cache->k_stride[2] >= cache->k_stride[1] || cache->v_stride[2] >= cache->v_stride[1];
    a.spread = many || apart || cache->dim > 128 ? 0 : a.heads % 4 == 0 ? 2 : a.heads % 2 == 0 ? 1 : 0;
    while (a.spread > 0 && requests * a.heads >> a.spread < 128)
        --a.spread;
    // no more workgroups than shares can be: row tiles times the blocks that the
    // table's width allows
    const int64_t blocks = (a.reach + gemv::kCostBlock - 1) / gemv::kCostBlock;
    int64_t tiles = tokens * a.group / gemv::kAttnRows + (requests < tokens ? requests : tokens);
    tiles = (tiles < tokens * a.group ? tiles : tokens * a.group) * a.heads; // at most tokens * q_heads, below 2^31
    const int64_t cap = (INT_MAX - 1) / tiles; // of a tile's cost
    const int64_t start = cache->dim == 64 ? 16 : 8;
    a.tile_cost = (int)(start <= cap / 2 ? start : cap > 1 ? cap / 2 : 1);
    while (a.tile_cost + (blocks >> a.unit_log2) > cap)
        ++a.unit_log2;
    const int64_t most = gemv::kAttnGroups, shares = (blocks + a.tile_cost) / 8 + 1;
    const int grid = (int)(tiles >= most || shares >= most || tiles * shares >= most ? most : tiles * shares);
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)grid), dim3(gemv::kThreads), args, 0,
                                         static_cast<hipStream_t>(hip_stream));
    return gemv::finish_launch((int)e);
}

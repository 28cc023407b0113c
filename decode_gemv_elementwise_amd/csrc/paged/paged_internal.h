// Shared by the paged operators' host checks (paged_validate.cpp) and their
// HIP translation units.  Host code only.
#pragma once

#include <cstdint>

#include "gemv_paged.h"

namespace gemv {

// n / d for 0 <= n < 2^31 as (mulhi(mul, n) + n) >> shift: mul is
// floor(2^32 (2^shift - d) / d) + 1 with shift = ceil(log2 d), and the sum
// stays below 2^32 because mulhi(mul, n) <= n.  A power of two gives mul = 1,
// whose high product is 0.
struct FastDiv {
    uint32_t mul, shift, d;
};

inline FastDiv fast_div(int64_t d)
{
    uint32_t s = 0;
    while ((1ll << s) < d)
        ++s;
    const uint64_t m = (((1ull << s) - (uint64_t)d) << 32) / (uint64_t)d + 1;
    return FastDiv{(uint32_t)m, s, (uint32_t)d};
}

constexpr int64_t kPagedMaxRequests = 1 << 20;

// The attention's workspace: a counter for every workgroup, then the parts, two
// places for every workgroup.  A part holds one workgroup's share of the keys of
// one row tile: the rows' sums over v, their maxima and their weight sums.
constexpr int kAttnRows = 16; // rows of a tile of few rows
constexpr int kAttnCounters = 2048;
constexpr int64_t kAttnGroups = 512; // workgroups of a launch: as many as the 256 compute units hold at once
// Floats of the largest part: 128 rows of up to 128 values (half as many of 256),
// and a maximum and a sum of each lane.
constexpr int64_t attn_part_floats(int64_t dim) { return 128 * (dim < 128 ? dim : 128) + 512; }

int validate_slots(const int32_t *cached, const int32_t *fresh, int64_t requests, const int32_t *free_pages,
                   int64_t num_free, int64_t page_size, int32_t *block_table, int64_t table_width,
                   int64_t table_stride, int64_t tokens, int32_t *query_start, int32_t *kv_len, int32_t *token_request,
                   int32_t *positions, int32_t *slots, int32_t *used);
int validate_append(const void *q, const void *k, const void *v, int src_type, int64_t tokens, int64_t q_heads,
                    int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions, int64_t axes,
                    const int32_t *axis, const float *inv_freq, int64_t rot, int style, const int32_t *slots,
                    const void *q_out, const gemv_kv_cache *cache);
int validate_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache *cache,
                  const int32_t *block_table, int64_t table_width, int64_t table_stride, const int32_t *query_start,
                  const int32_t *kv_len, int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                  int64_t sinks, const void *out, int out_type, int64_t out_token_stride, int64_t out_head_stride,
                  const void *workspace, int64_t workspace_bytes);
int64_t attn_workspace(int64_t dim);

// As in gemv_internal.h: records a launch's hipError_t for the calling thread.
int finish_launch(int hip_error);

} // namespace gemv

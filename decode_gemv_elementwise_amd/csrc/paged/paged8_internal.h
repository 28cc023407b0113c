// Shared by the host checks of the operators over a cache of 8-bit codes
// (paged8_validate.cpp) and their HIP translation units.  Host code only.
#pragma once

#include "gemv_paged8.h"
#include "paged_internal.h"

namespace gemv {

int validate_append8(const void *q, const void *k, const void *v, int src_type, int64_t tokens, int64_t q_heads,
                     int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions, int64_t axes,
                     const int32_t *axis, const float *inv_freq, int64_t rot, int style, const int32_t *slots,
                     const void *q_out, int q_out_type, const gemv_kv_cache8 *cache);
int validate_read8(const gemv_kv_cache8 *cache, const int32_t *slots, int64_t tokens, const void *k_out,
                   const void *v_out, int out_type, int64_t k_out_stride, int64_t v_out_stride);
int validate_attn8(const void *q, int q_type, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache8 *cache,
                   const int32_t *block_table, int64_t table_width, int64_t table_stride, const int32_t *query_start,
                   const int32_t *kv_len, int64_t requests, int64_t tokens, int64_t q_heads, float scale,
                   int64_t window, int64_t sinks, const void *out, int out_type, int64_t out_token_stride,
                   int64_t out_head_stride, const void *workspace, int64_t workspace_bytes);

// The attention's kernel for heads of that many values.  many: row tiles of many rows.
// runs: of few rows, that eight keys from a multiple of eight on lie in one page and share
// a scale; of many, that 16 lie in one page, and a block of 16 or more holds all or none
// of them, a shorter one divides 16.
const void *paged8_attn_kernel_64(int code, bool bf, bool f32out, bool runs, bool many);
const void *paged8_attn_kernel_128(int code, bool bf, bool f32out, bool runs, bool many);
const void *paged8_attn_kernel_256(int code, bool bf, bool f32out, bool runs, bool many);

} // namespace gemv

/*
 * gemv_paged.h -- C ABI of the paged key/value cache's operators for MI355X
 * (gfx950): what a decode layer runs between its qkv product and its output
 * product (gemv_fused.h).
 *
 *   gemv_paged_slots   block tables and slot maps from the requests' lengths
 *   gemv_paged_append  rotary positions for q and k; k and v into their pages
 *   gemv_paged_attn    attention of the new tokens over the paged cache
 *
 * They belong to the same library and keep its rules: the caller owns every
 * buffer, nothing is allocated, copied or synchronised, every check runs
 * before the launch and a rejected call launches nothing; calls are
 * asynchronous on the given HIP stream (NULL = the null stream) and may be
 * captured into a graph.  Status codes, gemv_strerror and
 * gemv_last_hip_error are those of gemv_fused.h.  Lengths, tables and slots
 * live in device memory and are read by the kernels only: the host never sees
 * them, so a captured step runs on for new lengths.  What the kernels read
 * from device memory they check themselves: a length, page id or slot that
 * points outside its buffer is dropped as stated below, never followed.
 *
 * Element types are GEMV_W_F32, GEMV_W_F16 and GEMV_W_BF16.
 */
#ifndef GEMV_PAGED_H
#define GEMV_PAGED_H

#include <stdint.h>

#include "gemv_fused.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A paged key/value cache in device memory.  Element e of key/value head h of
 * the token at place s of page b is k[b * k_stride[0] + s * k_stride[1] +
 * h * k_stride[2] + e], e < dim; the same for v.  Strides are in elements,
 * positive, multiples of 8 and below 2^31 each, and no two elements share an
 * address; k and v are 16-byte aligned.  Both orders in use, [page][token][head][dim]
 * and [page][head][token][dim], are strides of this form. */
typedef struct {
    void *k, *v;
    int32_t type;      /* GEMV_W_F16 or GEMV_W_BF16 */
    int32_t heads;     /* key/value heads, 1..GEMV_PAGED_MAX_HEADS */
    int32_t dim;       /* values per head */
    int32_t page_size; /* tokens per page, 1..GEMV_PAGED_MAX_PAGE */
    int64_t num_pages; /* >= 1; num_pages * page_size below 2^31 */
    int64_t k_stride[3], v_stride[3];
} gemv_kv_cache;

#define GEMV_PAGED_MAX_HEADS 4096
#define GEMV_PAGED_MAX_PAGE 65536
#define GEMV_PAGED_MAX_DIM 512 /* gemv_paged_append; gemv_paged_attn takes 64, 128 and 256 */

/* Block tables and slot maps, built from request lengths in one launch.
 * Request r < requests has cached[r] tokens in the cache and fresh[r] new ones
 * (a negative length counts as 0).  With P = page_size:
 *     start_r       = sum of fresh over the requests before r
 *     kv_len[r]     = cached[r] + fresh[r]
 *     old_r, new_r  = ceil(cached[r] / P), ceil(kv_len[r] / P)
 *     block_table[r][old_r .. new_r) = the next new_r - old_r ids of
 *                     free_pages, which the requests take in their order
 *     used[0]       = the ids that all requests need together
 *     query_start[r] = start_r, query_start[requests] = the sum
 * and for new token i of request r, t = start_r + i:
 *     token_request[t] = r, positions[t] = cached[r] + i,
 *     slots[t] = block_table[r][positions[t] / P] * P + positions[t] % P
 * Places t from the sum up to `tokens` hold token_request -1, positions 0 and
 * slots -1, so a step may be padded to a captured size.
 * Entries below old_r are read for the page that is still being filled and
 * otherwise left alone; entries from new_r on are left alone.
 * What does not fit: a request whose tokens run past `tokens` is cut there (its
 * fresh count is what is left); ids needed past num_free are -1 in the table
 * and give slots -1 (used[0] > num_free tells the host); pages past table_width
 * have no entry and give slots -1; so does a table entry that is negative or
 * whose slot would pass 2^31 - 1.
 *  cached, fresh   [requests] int32.
 *  free_pages      [num_free] int32; may be NULL when num_free is 0.
 *  block_table     [requests] rows of table_width int32, table_stride apart.
 *  query_start     [requests + 1]; kv_len [requests]; used [1] int32.
 *  token_request, positions, slots   [tokens] int32; may be NULL when tokens
 *                  is 0.
 * Outputs overlap neither the inputs nor one another (GEMV_E_ALIAS).
 * requests 1..2^20, tokens 0..2^31 - 1, table_width >= 1 (else GEMV_E_DIM). */
int gemv_paged_slots(const int32_t *cached, const int32_t *fresh, int64_t requests, const int32_t *free_pages,
                     int64_t num_free, int64_t page_size, int32_t *block_table, int64_t table_width,
                     int64_t table_stride, int64_t tokens, int32_t *query_start, int32_t *kv_len,
                     int32_t *token_request, int32_t *positions, int32_t *slots, int32_t *used, void *hip_stream);

/* The host-side checks of gemv_paged_slots; no HIP call. */
int gemv_paged_slots_validate(const int32_t *cached, const int32_t *fresh, int64_t requests, const int32_t *free_pages,
                              int64_t num_free, int64_t page_size, int32_t *block_table, int64_t table_width,
                              int64_t table_stride, int64_t tokens, int32_t *query_start, int32_t *kv_len,
                              int32_t *token_request, int32_t *positions, int32_t *slots, int32_t *used);

/* Pairing of a head's values by the rotation: pair i is (i, i + rot / 2) or
 * (2 i, 2 i + 1). */
typedef enum { GEMV_ROPE_HALVES = 0, GEMV_ROPE_PAIRS = 1 } gemv_rope_style;

/* Rotary positions and the write into the cache, one launch.  For token t and
 * pair i < rot / 2,
 *     angle = positions[axis[i]][t] * inv_freq[i]       (formed in 64 bits)
 *     (a, b) -> (a cos - b sin, b cos + a sin)          (in 32 bits)
 * over q and k of every head; the values from rot on pass unturned.  Then, with
 * each value rounded once to the cache's type, q goes to q_out and k and v to
 * place slots[t] % P of page slots[t] / P.  A slot that is negative or not
 * below num_pages * P writes no k and v (its q is still written); two tokens
 * of one slot leave either's values.
 *  q, k, v     rows of q_heads (cache->heads) times dim values of src_type, the
 *              rows q_stride, k_stride and v_stride elements apart: parts of one
 *              qkv row, or buffers of their own.
 *  positions   [axes][tokens] int32.  axes > 1 is for images and video (time,
 *              height, width): axis[i] int32 names the axis that turns pair i.
 *              A pair whose axis is outside 0..axes-1 is not turned.  axis may
 *              be NULL: every pair goes by axis 0.
 *  inv_freq    [rot / 2] f32; may be NULL when rot is 0.
 *  rot         even, 0..dim.
 *  slots       [tokens] int32.
 *  q_out       [tokens][q_heads][dim] of the cache's type, contiguous.
 *  cache       dim a multiple of 8, up to GEMV_PAGED_MAX_DIM.
 * q_out, k and v of the cache overlap no input and not one another.
 * Tensors may have any alignment of their element; 16-byte aligned rows with
 * strides of whole 16 bytes take the wide path.  tokens 0 launches nothing. */
int gemv_paged_append(const void *q, const void *k, const void *v, int src_type, int64_t tokens, int64_t q_heads,
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions, int64_t axes,
                      const int32_t *axis, const float *inv_freq, int64_t rot, int style, const int32_t *slots,
                      void *q_out, const gemv_kv_cache *cache, void *hip_stream);

/* The host-side checks of gemv_paged_append; no HIP call. */
int gemv_paged_append_validate(const void *q, const void *k, const void *v, int src_type, int64_t tokens,
                               int64_t q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               const int32_t *positions, int64_t axes, const int32_t *axis, const float *inv_freq,
                               int64_t rot, int style, const int32_t *slots, void *q_out, const gemv_kv_cache *cache);

/* Attention of every request's new tokens over its paged cache.  Request r's
 * tokens are rows query_start[r] .. query_start[r + 1] of q, n_r of them, and
 * are the last n_r of its kv_len[r] tokens: new token i is at position
 * p = kv_len[r] - n_r + i.  For query head h, whose keys are those of head
 * h / (q_heads / cache->heads),
 *     out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q.k_j)
 * over the keys j that the token sees: j <= p, and, where window > 0,
 * j > p - window or j < sinks (the first tokens, which stay visible), and
 * whose page id is in 0..num_pages-1: a page released behind a window has id
 * -1 in the table and is never read.  A row that sees no key (or only keys of
 * score -infinity) is zero.  Keys that a row does not see do not enter its
 * result, also where they hold infinities or NaN.
 *  q           rows of q_heads heads of dim values of the cache's type, token
 *              and head strides in elements; 16-byte aligned, strides
 *              multiples of 8.
 *  block_table [requests] rows of table_width int32, table_stride apart; keys
 *              past table_width pages, or from 2^31 - 64 on, are not visible.
 *  query_start [requests + 1] int32, rising, within 0..tokens (cut to that);
 *              rows of q that belong to no request leave out unwritten.
 *  kv_len      [requests] int32.
 *  q_heads     a multiple of cache->heads; dim 64, 128 or 256.
 *  window      0: none.  sinks is read only where window > 0.
 *  out         rows as q's, with strides of its own, of the cache's type or
 *              f32 (out_type); 16-byte aligned, strides multiples of 8.
 *              out may not overlap anything that is read.
 *  workspace   16-byte aligned scratch that holds the parts of rows whose keys
 *              are split over workgroups; all zero before its first use and
 *              used by one stream at a time, and left ready for the next call
 *              whatever its shapes.  gemv_paged_attn_workspace gives the size
 *              that is enough for any call; where it is too small for a call's
 *              parts (0 and NULL included) no row's keys are split.
 * Sums, the softmax's statistics and the parts are held in 32 bits; the
 * weights w_j are rounded to the cache's type for the product with v (where
 * out is f32 they are carried as two pieces of that type).  An infinity of v
 * whose weight is too small to be held beside the row's largest (binary16: below
 * 2^-38 of it) gives that infinity or NaN, by where in the row its key lies. */
int gemv_paged_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache *cache,
                    const int32_t *block_table, int64_t table_width, int64_t table_stride, const int32_t *query_start,
                    const int32_t *kv_len, int64_t requests, int64_t tokens, int64_t q_heads, float scale,
                    int64_t window, int64_t sinks, void *out, int out_type, int64_t out_token_stride,
                    int64_t out_head_stride, void *workspace, int64_t workspace_bytes, void *hip_stream);

/* The host-side checks of gemv_paged_attn; no HIP call. */
int gemv_paged_attn_validate(const void *q, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache *cache,
                             const int32_t *block_table, int64_t table_width, int64_t table_stride,
                             const int32_t *query_start, const int32_t *kv_len, int64_t requests, int64_t tokens,
                             int64_t q_heads, float scale, int64_t window, int64_t sinks, const void *out, int out_type,
                             int64_t out_token_stride, int64_t out_head_stride, const void *workspace,
                             int64_t workspace_bytes);

/* The workspace that is enough for gemv_paged_attn with heads of dim values
 * (any lengths), in bytes, or GEMV_E_DIM. */
int64_t gemv_paged_attn_workspace(int64_t dim);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_PAGED_H */

/*
 * gemv_paged8.h -- C ABI of the operators over a paged key/value cache held in
 * 8 bits for MI355X (gfx950): those of gemv_paged.h for a cache of half the
 * bytes.  Block tables and slot maps are the same (gemv_paged_slots).
 *
 *   gemv_paged8_append  rotary positions for q and k; k and v quantised into
 *                       their pages
 *   gemv_paged8_read    tokens of the cache in 16 or 32 bits
 *   gemv_paged8_attn    attention of the new tokens over the cache
 *
 * They keep the rules of gemv_paged.h: the caller owns every buffer, nothing is
 * allocated, copied or synchronised, every check runs before the launch (one a
 * call), lengths, tables and slots are read from device memory by the kernels
 * alone, and what they read there is checked and never followed out of a buffer.
 *
 * A block is `block` neighbouring places of a page.  Each block has, for each
 * key/value head and for k and v apart, one byte b that stands for the scale
 * 2^(b - 127); 255 stands for NaN.  A value is its code times its block's scale:
 *   GEMV_KV_INT8  whole numbers from -127 to 127 (a code of -128 is taken as it is)
 *   GEMV_KV_E4M3  a sign, 4 bits of exponent and 3 of significand, up to 448, no
 *                 infinities (the "fn" form)
 * Scales are powers of two so that a value is exact in 16 bits (bf16 always;
 * binary16 within its range) and a block whose scale grows keeps what it holds:
 * e4m3 codes lose nothing but steps below their smallest one, and an int8 value is
 * within one step of its block's last scale however often that grew, where free
 * scales would add half a step each time.  Values below 2^-118 may be taken as 0.
 */
#ifndef GEMV_PAGED8_H
#define GEMV_PAGED8_H

#include <stdint.h>

#include "gemv_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMV_KV_INT8 = 0, GEMV_KV_E4M3 = 1 } gemv_kv_code;

/* A paged key/value cache of one byte a value.  Codes lie as in gemv_kv_cache, with
 * strides in bytes: k[b * k_stride[0] + s * k_stride[1] + h * k_stride[2] + e].
 * Those strides are positive, multiples of 16 and below 2^31 each, no two codes
 * share an address, and k and v are 16-byte aligned.  The scale of place s of page
 * b and head h is k_scale[b * ks_stride[0] + s / block * ks_stride[1] + h *
 * ks_stride[2]], strides positive and below 2^31, no two scales at one address.  What
 * is appended to has no byte twice among the four: they lie apart, or in one buffer, k
 * and v (or the two scales) with the same strides a fixed step apart, codes and scales
 * with the same page stride, so that a page may carry its scales. */
typedef struct {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    int32_t code;      /* gemv_kv_code */
    int32_t heads;     /* key/value heads, 1..GEMV_PAGED_MAX_HEADS */
    int32_t dim;       /* values per head, a multiple of 16 up to GEMV_PAGED_MAX_DIM */
    int32_t page_size; /* tokens per page, 1..GEMV_PAGED_MAX_PAGE */
    int32_t block;     /* tokens of a scale, a divisor of page_size */
    int64_t num_pages; /* >= 1; num_pages * page_size below 2^31 */
    int64_t k_stride[3], v_stride[3], ks_stride[3], vs_stride[3];
} gemv_kv_cache8;

/* Rotary positions and the quantising write into the cache, one launch.  q, k and
 * v are turned as by gemv_paged_append; q goes to q_out, rounded once to
 * q_out_type (GEMV_W_F16 or GEMV_W_BF16).  k and v go in, unrounded after their
 * turn, at place slots[t] % page_size of page slots[t] / page_size.  Of the tokens
 * of this call in one block, one head, let a be the largest size and M = 127
 * (int8) or 448 (e4m3):
 *     b' = the least byte from 1 up with a <= M 2^(b' - 127); 255 where one of the
 *          values is an infinity or NaN
 *     b  = b' if the block's first place is among the tokens' (the block is begun
 *          anew, whatever it held), else max(b', the byte that it has)
 *     the block's other codes c become round(c 2^(old - b)), where b has grown
 *     c_t = round(x_t 2^(127 - b))   (to nearest, ties to even)
 * so an infinity or NaN makes its block and head NaN until the block is begun anew.
 * A slot that is negative or not below num_pages * page_size writes no k and v (its
 * q is still written).  Tokens of one call whose slots lie in one block are
 * neighbours in the call (in any order), as gemv_paged_slots lays them out; where
 * others lie between them, that block's values are unspecified.  Two tokens of one slot
 * leave, value by value, either's, and those of their block may be rounded twice.
 *  q, k, v, src_type, tokens, positions, axes, axis, inv_freq, rot, style, slots
 *              as for gemv_paged_append, tokens up to 2^30.
 *  q_out       [tokens][q_heads][dim], contiguous, 16-byte aligned.
 * q_out overlaps no input and no part of the cache, from first to last byte, and the
 * cache no input.
 * 16-byte aligned rows with strides of whole 16 bytes, rot a multiple of 16
 * (GEMV_ROPE_HALVES) or 8 (GEMV_ROPE_PAIRS), and blocks of at most 16 floor(1024 / dim)
 * tokens (256 at dim 64, 128 at 128, 64 at 256, 32 at 512) take the wide path; others are
 * many times slower.  A token that makes its block's scale grow pays for the whole block. */
int gemv_paged8_append(const void *q, const void *k, const void *v, int src_type, int64_t tokens, int64_t q_heads,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions, int64_t axes,
                       const int32_t *axis, const float *inv_freq, int64_t rot, int style, const int32_t *slots,
                       void *q_out, int q_out_type, const gemv_kv_cache8 *cache, void *hip_stream);

/* The host-side checks of gemv_paged8_append; no HIP call. */
int gemv_paged8_append_validate(const void *q, const void *k, const void *v, int src_type, int64_t tokens,
                                int64_t q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                const int32_t *positions, int64_t axes, const int32_t *axis, const float *inv_freq,
                                int64_t rot, int style, const int32_t *slots, const void *q_out, int q_out_type,
                                const gemv_kv_cache8 *cache);

/* Tokens of the cache back in 16 or 32 bits, one launch: row t of k_out and v_out
 * gets the values at slots[t], each rounded once to out_type (which changes none in
 * f32 and bf16, nor in f16 within its range), or zeros where slots[t] is negative
 * or not below num_pages * page_size.
 *  slots       [tokens] int32; tokens 0 launches nothing.
 *  out_type    GEMV_W_F32, GEMV_W_F16 or GEMV_W_BF16.
 *  k_out, v_out  rows of heads times dim values, k_out_stride and v_out_stride
 *              elements apart; 16-byte aligned, strides multiples of 8.  Either may
 *              be NULL: it is left out.
 * They overlap no input and not one another. */
int gemv_paged8_read(const gemv_kv_cache8 *cache, const int32_t *slots, int64_t tokens, void *k_out, void *v_out,
                     int out_type, int64_t k_out_stride, int64_t v_out_stride, void *hip_stream);

/* The host-side checks of gemv_paged8_read; no HIP call. */
int gemv_paged8_read_validate(const gemv_kv_cache8 *cache, const int32_t *slots, int64_t tokens, const void *k_out,
                              const void *v_out, int out_type, int64_t k_out_stride, int64_t v_out_stride);

/* Attention of every request's new tokens over its paged cache: gemv_paged_attn
 * with k_j and v_j the cache's values, and every argument as there but for
 *  q_type      GEMV_W_F16 or GEMV_W_BF16: q's, and out's where that is not f32.
 *  cache       dim 64, 128 or 256.
 *  workspace   that of gemv_paged_attn (gemv_paged_attn_workspace); one may serve both.
 * A value that q's type does not hold (only binary16 has such: past 65504 an infinity, below
 * 2^-14 fewer bits) enters as it is or rounded to that type, by what else is in the call: a
 * caller cannot know which.  With bf16 a part w_j v_j that is below 2^-117, the row's largest
 * weight taken as 1, may be taken as 0.  Wide paths are for blocks of whole multiples of 8
 * tokens (calls of few tokens a request) and for pages of whole multiples of 16 whose
 * blocks divide or are divided by 16 (calls of many); others find each key by itself. */
int gemv_paged8_attn(const void *q, int q_type, int64_t q_token_stride, int64_t q_head_stride,
                     const gemv_kv_cache8 *cache, const int32_t *block_table, int64_t table_width,
                     int64_t table_stride, const int32_t *query_start, const int32_t *kv_len, int64_t requests,
                     int64_t tokens, int64_t q_heads, float scale, int64_t window, int64_t sinks, void *out,
                     int out_type, int64_t out_token_stride, int64_t out_head_stride, void *workspace,
                     int64_t workspace_bytes, void *hip_stream);

/* The host-side checks of gemv_paged8_attn; no HIP call. */
int gemv_paged8_attn_validate(const void *q, int q_type, int64_t q_token_stride, int64_t q_head_stride,
                              const gemv_kv_cache8 *cache, const int32_t *block_table, int64_t table_width,
                              int64_t table_stride, const int32_t *query_start, const int32_t *kv_len,
                              int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                              int64_t sinks, const void *out, int out_type, int64_t out_token_stride,
                              int64_t out_head_stride, const void *workspace, int64_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* GEMV_PAGED8_H */

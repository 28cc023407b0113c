// Host-side argument checks of the operators over a cache of 8-bit codes: null
// pointers, sizes, types, strides, alignment and the overlap rules.  No HIP call and no
// dereference of a device pointer, so it runs on a machine without a GPU.
#include "paged8_internal.h"

#include <cmath>
#include <initializer_list>

#include "paged_check.h"

namespace gemv {
namespace {

// The codes of k and v, and the scales of both; what a page holds of each.
struct CacheSpans {
    Span k, v, ks, vs;
    uint64_t k_page, v_page, ks_page, vs_page;
};

// Two tensors of the same extents share no element: their spans are apart, or they lie
// within one buffer with the same strides, the second a fixed step from the first, and
// that step nests among the strides.
bool twins_apart(Span x, Span y, const int64_t *xs, const int64_t *ys, const int64_t *extent, int64_t row)
{
    if (!overlap(x, y))
        return true;
    const uintptr_t step = x.lo < y.lo ? y.lo - x.lo : x.lo - y.lo;
    for (int d = 0; d < 3; ++d)
        if (xs[d] != ys[d])
            return false;
    if (step == 0 || step > (uintptr_t)kInt)
        return false;
    const int64_t stride[4] = {xs[0], xs[1], xs[2], (int64_t)step};
    const int64_t extents[4] = {extent[0], extent[1], extent[2], 2};
    return strides_nest(stride, extents, 4, row);
}

// Codes and scales share no byte: their spans are apart, or a page carries its scales.
// Then both have the page's stride, and counted from a page's first code, modulo that
// stride, a page's scales lie behind its codes and before the next one's.
bool pages_apart(Span codes, Span scales, const int64_t *cs, const int64_t *ss, uint64_t codes_page, uint64_t scales_page)
{
    if (!overlap(codes, scales))
        return true;
    const uint64_t step = (uint64_t)cs[0];
    if (cs[0] != ss[0] || codes_page > step || scales_page > step || codes.hi == UINTPTR_MAX || scales.hi == UINTPTR_MAX)
        return false; // the last two: no real buffer
    const uint64_t off = scales.lo >= codes.lo ? (scales.lo - codes.lo) % step : step - 1 - (codes.lo - scales.lo - 1) % step;
    return off >= codes_page && off <= step - scales_page;
}

int check_cache8(const gemv_kv_cache8 *c, CacheSpans *spans)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale)
        return GEMV_E_NULL;
    if (c->code != GEMV_KV_INT8 && c->code != GEMV_KV_E4M3)
        return GEMV_E_FMT;
    if (c->heads < 1 || c->heads > GEMV_PAGED_MAX_HEADS || c->page_size < 1 || c->page_size > GEMV_PAGED_MAX_PAGE ||
        c->dim < 16 || c->dim > GEMV_PAGED_MAX_DIM || c->dim % 16 != 0 || c->block < 1 || c->block > c->page_size ||
        c->page_size % c->block != 0 || c->num_pages < 1 || c->num_pages > kInt || c->num_pages * c->page_size > kInt)
        return GEMV_E_DIM;
    const int64_t extent[3] = {c->num_pages, c->page_size, c->heads};
    const int64_t scales[3] = {c->num_pages, c->page_size / c->block, c->heads};
    for (const int64_t *s : {c->k_stride, c->v_stride}) {
        for (int d = 0; d < 3; ++d)
            if (s[d] < 1 || s[d] > kInt || (extent[d] > 1 && s[d] % 16 != 0))
                return GEMV_E_LAYOUT;
        if (!strides_nest(s, extent, 3, c->dim))
            return GEMV_E_LAYOUT;
    }
    for (const int64_t *s : {c->ks_stride, c->vs_stride}) {
        for (int d = 0; d < 3; ++d)
            if (s[d] < 1 || s[d] > kInt)
                return GEMV_E_LAYOUT;
        if (!strides_nest(s, scales, 3, 1))
            return GEMV_E_LAYOUT;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return GEMV_E_ALIGN;
    // from dimension `from` on; below 2^64: a sum of three products of 62 bits
    const auto bytes = [](const int64_t *s, const int64_t *n, int64_t row, int from) {
        uint64_t e = (uint64_t)row;
        for (int d = from; d < 3; ++d)
            e += (uint64_t)(n[d] - 1) * (uint64_t)s[d];
        return e;
    };
    const auto codes = [&](const int64_t *s, int from) { return bytes(s, extent, c->dim, from); };
    const auto of_scales = [&](const int64_t *s, int from) { return bytes(s, scales, 1, from); };
    *spans = CacheSpans{span_of(c->k, codes(c->k_stride, 0)),
                        span_of(c->v, codes(c->v_stride, 0)),
                        span_of(c->k_scale, of_scales(c->ks_stride, 0)),
                        span_of(c->v_scale, of_scales(c->vs_stride, 0)),
                        codes(c->k_stride, 1),
                        codes(c->v_stride, 1),
                        of_scales(c->ks_stride, 1),
                        of_scales(c->vs_stride, 1)};
    return GEMV_OK;
}

// What is written into the cache lands in one place each.
bool cache8_apart(const gemv_kv_cache8 *c, const CacheSpans &s)
{
    const int64_t extent[3] = {c->num_pages, c->page_size, c->heads};
    const int64_t scales[3] = {c->num_pages, c->page_size / c->block, c->heads};
    return twins_apart(s.k, s.v, c->k_stride, c->v_stride, extent, c->dim) &&
           twins_apart(s.ks, s.vs, c->ks_stride, c->vs_stride, scales, 1) &&
           pages_apart(s.k, s.ks, c->k_stride, c->ks_stride, s.k_page, s.ks_page) &&
           pages_apart(s.k, s.vs, c->k_stride, c->vs_stride, s.k_page, s.vs_page) &&
           pages_apart(s.v, s.ks, c->v_stride, c->ks_stride, s.v_page, s.ks_page) &&
           pages_apart(s.v, s.vs, c->v_stride, c->vs_stride, s.v_page, s.vs_page);
}

} // namespace

int validate_append8(const void *q, const void *k, const void *v, int src_type, int64_t tokens, int64_t q_heads,
                     int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions, int64_t axes,
                     const int32_t *axis, const float *inv_freq, int64_t rot, int style, const int32_t *slots,
                     const void *q_out, int q_out_type, const gemv_kv_cache8 *cache)
{
    if (!cache || (tokens > 0 && (!q || !k || !v || !slots || !q_out || (rot > 0 && (!positions || !inv_freq)))))
        return GEMV_E_NULL;
    CacheSpans c;
    const int st = check_cache8(cache, &c);
    if (st != GEMV_OK)
        return st;
    if (!is_type(src_type) || (q_out_type != GEMV_W_F16 && q_out_type != GEMV_W_BF16))
        return GEMV_E_FMT;
    if (style != GEMV_ROPE_HALVES && style != GEMV_ROPE_PAIRS)
        return GEMV_E_ACT;
    if (tokens < 0 || tokens > kInt / 2 + 1 || q_heads < 1 || q_heads > GEMV_PAGED_MAX_HEADS || axes < 1 || axes > 64 ||
        rot < 0 || rot > cache->dim || rot % 2 != 0)
        return GEMV_E_DIM;
    const int64_t qrow = q_heads * cache->dim, krow = (int64_t)cache->heads * cache->dim;
    if (q_stride < 0 || q_stride > kInt || k_stride < 0 || k_stride > kInt || v_stride < 0 || v_stride > kInt)
        return GEMV_E_LAYOUT;
    const int64_t size = type_size(src_type);
    if (!aligned(q, size) || !aligned(k, size) || !aligned(v, size) || !aligned(positions, 4) || !aligned(axis, 4) ||
        !aligned(inv_freq, 4) || !aligned(slots, 4) || !aligned(q_out, 16))
        return GEMV_E_ALIGN;
    const Span ins[] = {span_of(q, strided_bytes(tokens, q_stride, qrow, size)),
                        span_of(k, strided_bytes(tokens, k_stride, krow, size)),
                        span_of(v, strided_bytes(tokens, v_stride, krow, size)),
                        span_of(positions, rot > 0 ? (uint64_t)axes * (uint64_t)tokens * 4 : 0),
                        span_of(axis, axis ? (uint64_t)rot * 2 : 0),
                        span_of(inv_freq, (uint64_t)rot * 2),
                        span_of(slots, (uint64_t)tokens * 4),
                        span_of(q_out, (uint64_t)tokens * (uint64_t)qrow * 2)};
    if (any_overlap(&ins[7], 1, ins, 7) || !cache8_apart(cache, c))
        return GEMV_E_ALIAS;
    for (const Span &s : {c.k, c.v, c.ks, c.vs})
        if (any_overlap(&s, 1, ins, 8))
            return GEMV_E_ALIAS;
    return GEMV_OK;
}

int validate_read8(const gemv_kv_cache8 *cache, const int32_t *slots, int64_t tokens, const void *k_out,
                   const void *v_out, int out_type, int64_t k_out_stride, int64_t v_out_stride)
{
    if (!cache || (tokens > 0 && (!slots || (!k_out && !v_out))))
        return GEMV_E_NULL;
    CacheSpans c;
    const int st = check_cache8(cache, &c);
    if (st != GEMV_OK)
        return st;
    if (!is_type(out_type))
        return GEMV_E_FMT;
    if (tokens < 0 || tokens > kInt)
        return GEMV_E_DIM;
    const int64_t row = (int64_t)cache->heads * cache->dim;
    for (const int64_t s : {k_out ? k_out_stride : row, v_out ? v_out_stride : row})
        if (s < 0 || s > kInt || (tokens > 1 && (s % 8 != 0 || s < row)))
            return GEMV_E_LAYOUT;
    if (!aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return GEMV_E_ALIGN;
    const int64_t size = type_size(out_type);
    const Span ins[] = {c.k, c.v, c.ks, c.vs, span_of(slots, (uint64_t)tokens * 4)};
    const Span outs[] = {span_of(k_out, k_out ? strided_bytes(tokens, k_out_stride, row, size) : 0),
                         span_of(v_out, v_out ? strided_bytes(tokens, v_out_stride, row, size) : 0)};
    return any_overlap(outs, 2, ins, 5) ? GEMV_E_ALIAS : GEMV_OK;
}

int validate_attn8(const void *q, int q_type, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache8 *cache,
                   const int32_t *block_table, int64_t table_width, int64_t table_stride, const int32_t *query_start,
                   const int32_t *kv_len, int64_t requests, int64_t tokens, int64_t q_heads, float scale,
                   int64_t window, int64_t sinks, const void *out, int out_type, int64_t out_token_stride,
                   int64_t out_head_stride, const void *workspace, int64_t workspace_bytes)
{
    if (!cache || !block_table || !query_start || !kv_len || (tokens > 0 && (!q || !out)) ||
        (workspace_bytes > 0 && !workspace))
        return GEMV_E_NULL;
    CacheSpans c;
    const int st = check_cache8(cache, &c);
    if (st != GEMV_OK)
        return st;
    if ((q_type != GEMV_W_F16 && q_type != GEMV_W_BF16) || (out_type != q_type && out_type != GEMV_W_F32))
        return GEMV_E_FMT;
    if (cache->dim != 64 && cache->dim != 128 && cache->dim != 256)
        return GEMV_E_DIM;
    if (requests < 1 || requests > kPagedMaxRequests || tokens < 0 || tokens > kInt || table_width < 1 ||
        table_width > kInt || q_heads < 1 || q_heads > GEMV_PAGED_MAX_HEADS || q_heads % cache->heads != 0 ||
        tokens * q_heads > kInt || window < 0 || window > kInt || sinks < 0 || sinks > kInt || workspace_bytes < 0 ||
        !std::isfinite(scale))
        return GEMV_E_DIM;
    if (table_stride < (requests > 1 ? table_width : 1) || table_stride > kInt)
        return GEMV_E_LAYOUT;
    const int64_t qs[2] = {q_token_stride, q_head_stride}, os[2] = {out_token_stride, out_head_stride};
    const int64_t extent[2] = {tokens, q_heads};
    for (int d = 0; d < 2; ++d)
        if (qs[d] < 0 || qs[d] > kInt || os[d] < 0 || os[d] > kInt ||
            (extent[d] > 1 && (qs[d] % 8 != 0 || os[d] % 8 != 0 || os[d] == 0)))
            return GEMV_E_LAYOUT;
    if (tokens > 0 && !strides_nest(os, extent, 2, cache->dim))
        return GEMV_E_LAYOUT;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(block_table, 4) ||
        !aligned(query_start, 4) || !aligned(kv_len, 4))
        return GEMV_E_ALIGN;
    const auto rows = [&](const int64_t *s, int64_t size) -> uint64_t {
        return tokens == 0 ? 0
                           : bytes_of((uint64_t)(tokens - 1) * (uint64_t)s[0] +
                                          (uint64_t)(q_heads - 1) * (uint64_t)s[1] + (uint64_t)cache->dim,
                                      size);
    };
    const Span ins[] = {span_of(q, rows(qs, 2)), c.k, c.v, c.ks, c.vs,
                        span_of(block_table, strided_bytes(requests, table_stride, table_width, 4)),
                        span_of(query_start, (uint64_t)requests * 4 + 4), span_of(kv_len, (uint64_t)requests * 4)};
    const Span outs[] = {span_of(out, rows(os, type_size(out_type))), span_of(workspace, (uint64_t)workspace_bytes)};
    return any_overlap(outs, 2, ins, 8) ? GEMV_E_ALIAS : GEMV_OK;
}

} // namespace gemv

extern "C" {

int gemv_paged8_append_validate(const void *q, const void *k, const void *v, int src_type, int64_t tokens,
                                int64_t q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                const int32_t *positions, int64_t axes, const int32_t *axis, const float *inv_freq,
                                int64_t rot, int style, const int32_t *slots, const void *q_out, int q_out_type,
                                const gemv_kv_cache8 *cache)
{
    return gemv::validate_append8(q, k, v, src_type, tokens, q_heads, q_stride, k_stride, v_stride, positions, axes,
                                  axis, inv_freq, rot, style, slots, q_out, q_out_type, cache);
}

int gemv_paged8_read_validate(const gemv_kv_cache8 *cache, const int32_t *slots, int64_t tokens, const void *k_out,
                              const void *v_out, int out_type, int64_t k_out_stride, int64_t v_out_stride)
{
    return gemv::validate_read8(cache, slots, tokens, k_out, v_out, out_type, k_out_stride, v_out_stride);
}

int gemv_paged8_attn_validate(const void *q, int q_type, int64_t q_token_stride, int64_t q_head_stride,
                              const gemv_kv_cache8 *cache, const int32_t *block_table, int64_t table_width,
                              int64_t table_stride, const int32_t *query_start, const int32_t *kv_len,
                              int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                              int64_t sinks, const void *out, int out_type, int64_t out_token_stride,
                              int64_t out_head_stride, const void *workspace, int64_t workspace_bytes)
{
    return gemv::validate_attn8(q, q_type, q_token_stride, q_head_stride, cache, block_table, table_width, table_stride,
                                query_start, kv_len, requests, tokens, q_heads, scale, window, sinks, out, out_type,
                                out_token_stride, out_head_stride, workspace, workspace_bytes);
}

} // extern "C"

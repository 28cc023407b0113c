// Host-side argument checks of the paged operators: null pointers, sizes,
// types, strides, alignment and the overlap rules.  No HIP call and no
// dereference of a device pointer, so it runs on a machine without a GPU.
#include "paged_internal.h"

#include <climits>
#include <cmath>
#include <initializer_list>

namespace gemv {
namespace {

constexpr int64_t kInt = INT32_MAX;

struct Span {
    uintptr_t lo, hi; // [lo, hi)
};

bool overlap(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }

// A span past the top of the address space is no real buffer: it is widened to
// the whole space, so that it overlaps every other and the call is rejected.
Span span_of(const void *p, uint64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (bytes > UINTPTR_MAX - lo)
        return Span{0, UINTPTR_MAX};
    return Span{lo, lo + bytes};
}

// Any output over any input, or over another output.
bool any_overlap(const Span *outs, int nouts, const Span *ins, int nins)
{
    for (int i = 0; i < nouts; ++i) {
        for (int j = 0; j < nins; ++j)
            if (overlap(outs[i], ins[j]))
                return true;
        for (int j = i + 1; j < nouts; ++j)
            if (overlap(outs[i], outs[j]))
                return true;
    }
    return false;
}

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_type(int t) { return t == GEMV_W_F32 || t == GEMV_W_F16 || t == GEMV_W_BF16; }

int64_t type_size(int t) { return t == GEMV_W_F32 ? 4 : 2; }

// Elements to bytes; a product past 64 bits is the whole address space.
uint64_t bytes_of(uint64_t elements, int64_t size)
{
    return elements > UINT64_MAX / (uint64_t)size ? UINT64_MAX : elements * (uint64_t)size;
}

// Bytes from the first row's start to the last row's end.  Strides and extents
// that reach here are below 2^31 each.
uint64_t strided_bytes(int64_t rows, int64_t stride, int64_t row, int64_t size)
{
    return rows == 0 ? 0 : bytes_of((uint64_t)(rows - 1) * (uint64_t)stride + (uint64_t)row, size);
}

// The strides (n up to 4) nest without two elements meeting: taken from the
// smallest up, each is at least what those below it span.
bool strides_nest(const int64_t *stride, const int64_t *extent, int n, int64_t row)
{
    bool done[4] = {false, false, false, false};
    int64_t reach = row; // elements that the dimensions taken so far span
    for (int i = 0; i < n; ++i) {
        int best = -1;
        for (int d = 0; d < n; ++d)
            if (!done[d] && (best < 0 || stride[d] < stride[best] ||
                             (stride[d] == stride[best] && extent[d] < extent[best])))
                best = d;
        done[best] = true;
        if (extent[best] == 1)
            continue;
        if (stride[best] < reach)
            return false;
        reach += (extent[best] - 1) * stride[best]; // one extent is up to 2^31, the others far smaller: below 2^63
    }
    return true;
}

int check_cache(const gemv_kv_cache *c, Span *k, Span *v)
{
    if (!c || !c->k || !c->v)
        return GEMV_E_NULL;
    if (c->type != GEMV_W_F16 && c->type != GEMV_W_BF16)
        return GEMV_E_FMT;
    if (c->heads < 1 || c->heads > GEMV_PAGED_MAX_HEADS || c->page_size < 1 || c->page_size > GEMV_PAGED_MAX_PAGE ||
        c->dim < 8 || c->dim > GEMV_PAGED_MAX_DIM || c->dim % 8 != 0 || c->num_pages < 1 || c->num_pages > kInt ||
        c->num_pages * c->page_size > kInt)
        return GEMV_E_DIM;
    const int64_t extent[3] = {c->num_pages, c->page_size, c->heads};
    for (const int64_t *s : {c->k_stride, c->v_stride}) {
        for (int d = 0; d < 3; ++d)
            if (s[d] < 1 || s[d] > kInt || (extent[d] > 1 && s[d] % 8 != 0))
                return GEMV_E_LAYOUT;
        if (!strides_nest(s, extent, 3, c->dim))
            return GEMV_E_LAYOUT;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16))
        return GEMV_E_ALIGN;
    auto bytes = [&](const int64_t *s) {
        uint64_t e = (uint64_t)c->dim;
        for (int d = 0; d < 3; ++d)
            e += (uint64_t)(extent[d] - 1) * (uint64_t)s[d];
        return bytes_of(e, 2);
    };
    *k = span_of(c->k, bytes(c->k_stride));
    *v = span_of(c->v, bytes(c->v_stride));
    return GEMV_OK;
}

// k and v of one cache share no element: their spans are apart, or they lie
// within one buffer with the same strides, v a fixed step from k, and that step
// nests among the strides (a buffer [page][2][token][head][dim], for one).
bool kv_apart(const gemv_kv_cache *c, Span k, Span v)
{
    if (!overlap(k, v))
        return true;
    const uintptr_t step = k.lo < v.lo ? v.lo - k.lo : k.lo - v.lo;
    for (int d = 0; d < 3; ++d)
        if (c->k_stride[d] != c->v_stride[d])
            return false;
    if (step == 0 || step / 2 > (uintptr_t)kInt)
        return false;
    const int64_t stride[4] = {c->k_stride[0], c->k_stride[1], c->k_stride[2], (int64_t)(step / 2)};
    const int64_t extent[4] = {c->num_pages, c->page_size, c->heads, 2};
    return strides_nest(stride, extent, 4, c->dim);
}

} // namespace

int validate_slots(const int32_t *cached, const int32_t *fresh, int64_t requests, const int32_t *free_pages,
                   int64_t num_free, int64_t page_size, int32_t *block_table, int64_t table_width,
                   int64_t table_stride, int64_t tokens, int32_t *query_start, int32_t *kv_len, int32_t *token_request,
                   int32_t *positions, int32_t *slots, int32_t *used)
{
    if (!cached || !fresh || !block_table || !query_start || !kv_len || !used || (num_free > 0 && !free_pages) ||
        (tokens > 0 && (!token_request || !positions || !slots)))
        return GEMV_E_NULL;
    if (requests < 1 || requests > kPagedMaxRequests || num_free < 0 || num_free > kInt || page_size < 1 ||
        page_size > GEMV_PAGED_MAX_PAGE || table_width < 1 || table_width > kInt || tokens < 0 || tokens > kInt)
        return GEMV_E_DIM;
    if (table_stride < (requests > 1 ? table_width : 1) || table_stride > kInt)
        return GEMV_E_LAYOUT;
    for (const void *p : {(const void *)cached, (const void *)fresh, (const void *)free_pages, (const void *)block_table,
                          (const void *)query_start, (const void *)kv_len, (const void *)token_request,
                          (const void *)positions, (const void *)slots, (const void *)used})
        if (!aligned(p, 4))
            return GEMV_E_ALIGN;
    const uint64_t r = (uint64_t)requests * 4, t = (uint64_t)tokens * 4;
    const Span ins[] = {span_of(cached, r), span_of(fresh, r), span_of(free_pages, (uint64_t)num_free * 4)};
    const Span outs[] = {span_of(block_table, strided_bytes(requests, table_stride, table_width, 4)),
                         span_of(query_start, r + 4), span_of(kv_len, r), span_of(token_request, t),
                         span_of(positions, t), span_of(slots, t), span_of(used, 4)};
    return any_overlap(outs, 7, ins, 3) ? GEMV_E_ALIAS : GEMV_OK;
}

int validate_append(const void *q, const void *k, const void *v, int src_type, int64_t tokens, int64_t q_heads,
                    int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t *positions, int64_t axes,
                    const int32_t *axis, const float *inv_freq, int64_t rot, int style, const int32_t *slots,
                    const void *q_out, const gemv_kv_cache *cache)
{
    if (!cache || (tokens > 0 && (!q || !k || !v || !slots || !q_out || (rot > 0 && (!positions || !inv_freq)))))
        return GEMV_E_NULL;
    Span ck, cv;
    int st = check_cache(cache, &ck, &cv);
    if (st != GEMV_OK)
        return st;
    if (!is_type(src_type))
        return GEMV_E_FMT;
    if (style != GEMV_ROPE_HALVES && style != GEMV_ROPE_PAIRS)
        return GEMV_E_ACT;
    if (tokens < 0 || tokens > kInt || q_heads < 1 || q_heads > GEMV_PAGED_MAX_HEADS || axes < 1 || axes > 64 ||
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
                        span_of(slots, (uint64_t)tokens * 4)};
    const Span outs[] = {span_of(q_out, (uint64_t)tokens * (uint64_t)qrow * 2)};
    const Span ck1[] = {ck}, cv1[] = {cv};
    if (any_overlap(outs, 1, ins, 7) || any_overlap(outs, 1, ck1, 1) || any_overlap(outs, 1, cv1, 1) ||
        any_overlap(ck1, 1, ins, 7) || any_overlap(cv1, 1, ins, 7) || !kv_apart(cache, ck, cv))
        return GEMV_E_ALIAS;
    return GEMV_OK;
}

int validate_attn(const void *q, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache *cache,
                  const int32_t *block_table, int64_t table_width, int64_t table_stride, const int32_t *query_start,
                  const int32_t *kv_len, int64_t requests, int64_t tokens, int64_t q_heads, float scale, int64_t window,
                  int64_t sinks, const void *out, int out_type, int64_t out_token_stride, int64_t out_head_stride,
                  const void *workspace, int64_t workspace_bytes)
{
    if (!cache || !block_table || !query_start || !kv_len || (tokens > 0 && (!q || !out)) ||
        (workspace_bytes > 0 && !workspace))
        return GEMV_E_NULL;
    Span ck, cv;
    int st = check_cache(cache, &ck, &cv);
    if (st != GEMV_OK)
        return st;
    if (out_type != cache->type && out_type != GEMV_W_F32)
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
    auto rows = [&](const int64_t *s, int64_t size) -> uint64_t {
        return tokens == 0 ? 0
                           : bytes_of((uint64_t)(tokens - 1) * (uint64_t)s[0] +
                                          (uint64_t)(q_heads - 1) * (uint64_t)s[1] + (uint64_t)cache->dim,
                                      size);
    };
    const Span ins[] = {span_of(q, rows(qs, 2)), ck, cv,
                        span_of(block_table, strided_bytes(requests, table_stride, table_width, 4)),
                        span_of(query_start, (uint64_t)requests * 4 + 4), span_of(kv_len, (uint64_t)requests * 4)};
    const Span outs[] = {span_of(out, rows(os, type_size(out_type))), span_of(workspace, (uint64_t)workspace_bytes)};
    return any_overlap(outs, 2, ins, 6) ? GEMV_E_ALIAS : GEMV_OK;
}

int64_t attn_workspace(int64_t dim)
{
    if (dim != 64 && dim != 128 && dim != 256)
        return GEMV_E_DIM;
    return kAttnCounters * 4 + 2 * kAttnGroups * attn_part_floats(dim) * 4;
}

} // namespace gemv

extern "C" {

int gemv_paged_slots_validate(const int32_t *cached, const int32_t *fresh, int64_t requests, const int32_t *free_pages,
                              int64_t num_free, int64_t page_size, int32_t *block_table, int64_t table_width,
                              int64_t table_stride, int64_t tokens, int32_t *query_start, int32_t *kv_len,
                              int32_t *token_request, int32_t *positions, int32_t *slots, int32_t *used)
{
    return gemv::validate_slots(cached, fresh, requests, free_pages, num_free, page_size, block_table, table_width,
                                table_stride, tokens, query_start, kv_len, token_request, positions, slots, used);
}

int gemv_paged_append_validate(const void *q, const void *k, const void *v, int src_type, int64_t tokens,
                               int64_t q_heads, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               const int32_t *positions, int64_t axes, const int32_t *axis, const float *inv_freq,
                               int64_t rot, int style, const int32_t *slots, void *q_out, const gemv_kv_cache *cache)
{
    return gemv::validate_append(q, k, v, src_type, tokens, q_heads, q_stride, k_stride, v_stride, positions, axes, axis,
                                 inv_freq, rot, style, slots, q_out, cache);
}

int gemv_paged_attn_validate(const void *q, int64_t q_token_stride, int64_t q_head_stride, const gemv_kv_cache *cache,
                             const int32_t *block_table, int64_t table_width, int64_t table_stride,
                             const int32_t *query_start, const int32_t *kv_len, int64_t requests, int64_t tokens,
                             int64_t q_heads, float scale, int64_t window, int64_t sinks, const void *out, int out_type,
                             int64_t out_token_stride, int64_t out_head_stride, const void *workspace,
                             int64_t workspace_bytes)
{
    return gemv::validate_attn(q, q_token_stride, q_head_stride, cache, block_table, table_width, table_stride,
                               query_start, kv_len, requests, tokens, q_heads, scale, window, sinks, out, out_type,
                               out_token_stride, out_head_stride, workspace, workspace_bytes);
}

int64_t gemv_paged_attn_workspace(int64_t dim) { return gemv::attn_workspace(dim); }

} // extern "C"

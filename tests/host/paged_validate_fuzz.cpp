// Randomised checks of the paged operators' host checks (paged_validate.cpp),
// built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_paged_sanitize.py: extreme and negative sizes and strides, null,
// unaligned, overlapping and wrapping pointers.  A status is a documented one, a
// second identical call returns the same, and of an accepted call no output's
// bytes (counted here in 128 bits, first to last) meet an input's or run past the
// top of the address space.  Exits 1 on the first violation.
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "gemv_paged.h"

namespace {

typedef unsigned __int128 u128;

struct Rng {
    uint64_t s;
    uint64_t next()
    {
        uint64_t z = (s += 0x9E3779B97F4A7C15ull);
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
        z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
        return z ^ (z >> 31);
    }
    int64_t range(int64_t lo, int64_t hi) { return lo + (int64_t)(next() % (uint64_t)(hi - lo + 1)); }
    bool coin(int pct) { return (int64_t)(next() % 100) < pct; }
};

int64_t size_of(Rng &r, int64_t usual)
{
    static const int64_t edge[] = {0, -1, 1, 2, 7, 8, 64, 4096, 65536, 65537, (1LL << 31) - 8, (1LL << 31) - 1, 1LL << 31,
                                   1LL << 40, INT64_MAX, INT64_MIN};
    return r.coin(12) ? edge[r.next() % (sizeof(edge) / sizeof(edge[0]))] : r.coin(30) ? r.range(1, 40) : usual;
}

template <class T> T *address(Rng &r, int i)
{
    if (r.coin(2))
        return nullptr;
    if (r.coin(2))
        return reinterpret_cast<T *>(UINTPTR_MAX - (uintptr_t)r.range(0, 4096));
    uintptr_t a = 0x10000000u + 0x4000000u * (uintptr_t)(r.coin(10) ? r.range(0, 11) : i);
    if (r.coin(5))
        a += (uintptr_t)r.range(1, 15);
    return reinterpret_cast<T *>(a);
}

struct Span {
    u128 lo, hi;
};

Span span(const void *p, u128 bytes) { return Span{(u128)(uintptr_t)p, (u128)(uintptr_t)p + bytes}; }

void require(bool ok, const char *what, long i)
{
    if (!ok) {
        std::printf("violation in call %ld: %s\n", i, what);
        std::exit(1);
    }
}

void apart(const Span *outs, int no, const Span *ins, int ni, const char *what, long call)
{
    const u128 top = (u128)UINTPTR_MAX + 1;
    for (int i = 0; i < no; ++i) {
        require(outs[i].lo == outs[i].hi || outs[i].hi <= top, what, call);
        for (int j = 0; j < ni; ++j)
            require(outs[i].lo == outs[i].hi || ins[j].lo == ins[j].hi || outs[i].hi <= ins[j].lo || ins[j].hi <= outs[i].lo,
                    what, call);
    }
}

gemv_kv_cache cache(Rng &r, int i)
{
    gemv_kv_cache c{};
    c.k = address<void>(r, i);
    c.v = address<void>(r, i + 1);
    c.type = (int)r.range(r.coin(90) ? 1 : -1, r.coin(90) ? 2 : 4);
    c.heads = (int32_t)size_of(r, 2);
    c.dim = (int32_t)(r.coin(70) ? 64 << r.range(0, 2) : size_of(r, 8));
    c.page_size = (int32_t)size_of(r, 16);
    c.num_pages = size_of(r, 10);
    const bool hnd = r.coin(50);
    const int64_t s[3] = {(int64_t)((uint64_t)c.page_size * (uint64_t)c.heads * (uint64_t)c.dim),
                          hnd ? c.dim : (int64_t)((uint64_t)c.heads * (uint64_t)c.dim),
                          hnd ? (int64_t)((uint64_t)c.page_size * (uint64_t)c.dim) : c.dim};
    for (int d = 0; d < 3; ++d) {
        c.k_stride[d] = r.coin(5) ? size_of(r, 64) : s[d];
        c.v_stride[d] = r.coin(5) ? size_of(r, 64) : s[d];
    }
    return c;
}

u128 cache_bytes(const gemv_kv_cache &c, const int64_t *s)
{
    return 2 * ((u128)(c.num_pages - 1) * s[0] + (u128)(c.page_size - 1) * s[1] + (u128)(c.heads - 1) * s[2] + c.dim);
}

bool known(int st) { return st <= 0 && st > -64; }

} // namespace

int main(int argc, char **argv)
{
    const long n = argc > 1 ? std::atol(argv[1]) : 100000;
    Rng r{12345};
    long accepted[3] = {0, 0, 0};
    for (long i = 0; i < n; ++i) {
        {
            auto *cached = address<int32_t>(r, 0), *fresh = address<int32_t>(r, 1), *free_pages = address<int32_t>(r, 2),
                 *table = address<int32_t>(r, 3), *start = address<int32_t>(r, 4), *kv = address<int32_t>(r, 5),
                 *req = address<int32_t>(r, 6), *pos = address<int32_t>(r, 7), *map = address<int32_t>(r, 8),
                 *used = address<int32_t>(r, 9);
            const int64_t requests = size_of(r, 9), nfree = size_of(r, 50), page = size_of(r, 16), width = size_of(r, 12),
                          stride = size_of(r, 16), tokens = size_of(r, 33);
            auto call = [&] {
                return gemv_paged_slots_validate(cached, fresh, requests, free_pages, nfree, page, table, width, stride, tokens,
                                                 start, kv, req, pos, map, used);
            };
            const int st = call();
            require(known(st) && st == call(), "slots status", i);
            if (st == GEMV_OK) {
                ++accepted[0];
                const Span ins[] = {span(cached, (u128)requests * 4), span(fresh, (u128)requests * 4),
                                    span(free_pages, (u128)nfree * 4)};
                const Span outs[] = {span(table, 4 * ((u128)(requests - 1) * stride + width)),
                                     span(start, ((u128)requests + 1) * 4), span(kv, (u128)requests * 4),
                                     span(req, (u128)tokens * 4), span(pos, (u128)tokens * 4), span(map, (u128)tokens * 4),
                                     span(used, 4)};
                apart(outs, 7, ins, 3, "slots buffers", i);
            }
        }
        {
            const gemv_kv_cache c = cache(r, 6);
            const int type = (int)r.range(0, r.coin(95) ? 2 : 5), style = (int)r.range(0, r.coin(95) ? 1 : 3);
            const int64_t size = type == 0 ? 4 : 2;
            auto *q = address<char>(r, 0), *k = address<char>(r, 1), *v = address<char>(r, 2);
            auto *pos = address<int32_t>(r, 3), *axis = r.coin(50) ? nullptr : address<int32_t>(r, 4), *map = address<int32_t>(r, 9);
            auto *inv = address<float>(r, 5);
            void *out = address<void>(r, 8);
            const int64_t tokens = size_of(r, 20), heads = size_of(r, 4), axes = size_of(r, 2), rot = size_of(r, 32);
            const int64_t qs = size_of(r, 1024), ks = size_of(r, 512), vs = size_of(r, 512);
            auto call = [&] {
                return gemv_paged_append_validate(q, k, v, type, tokens, heads, qs, ks, vs, pos, axes, axis, inv, rot, style,
                                                  map, out, &c);
            };
            const int st = call();
            require(known(st) && st == call(), "append status", i);
            if (st == GEMV_OK && tokens > 0) {
                ++accepted[1];
                const u128 t = (u128)(tokens - 1);
                const Span ins[] = {span(q, (t * qs + (u128)heads * c.dim) * size),
                                    span(k, (t * ks + (u128)c.heads * c.dim) * size),
                                    span(v, (t * vs + (u128)c.heads * c.dim) * size),
                                    span(pos, rot > 0 ? (u128)axes * tokens * 4 : 0), span(axis, axis ? (u128)rot * 2 : 0),
                                    span(inv, (u128)rot * 2), span(map, (u128)tokens * 4)};
                const Span outs[] = {span(out, (u128)tokens * heads * c.dim * 2), span(c.k, cache_bytes(c, c.k_stride)),
                                     span(c.v, cache_bytes(c, c.v_stride))};
                apart(outs, 3, ins, 7, "append buffers", i);
            }
        }
        {
            const gemv_kv_cache c = cache(r, 6);
            const int type = r.coin(90) ? (r.coin(50) ? 0 : c.type) : (int)r.range(-1, 5);
            auto *q = address<char>(r, 0), *out = address<char>(r, 1), *work = address<char>(r, 2);
            auto *table = address<int32_t>(r, 3), *start = address<int32_t>(r, 4), *kv = address<int32_t>(r, 5);
            const int64_t width = size_of(r, 12), stride = size_of(r, 16), requests = size_of(r, 9), tokens = size_of(r, 20),
                          heads = size_of(r, 4), window = size_of(r, 100), sinks = size_of(r, 4), bytes = size_of(r, 4096);
            const int64_t qt = size_of(r, 1024), qh = size_of(r, 256), ot = size_of(r, 1024), oh = size_of(r, 256);
            auto call = [&] {
                return gemv_paged_attn_validate(q, qt, qh, &c, table, width, stride, start, kv, requests, tokens, heads, 0.1f,
                                                window, sinks, out, type, ot, oh, work, bytes);
            };
            const int st = call();
            require(known(st) && st == call(), "attn status", i);
            if (st == GEMV_OK && tokens > 0) {
                ++accepted[2];
                const u128 t = (u128)(tokens - 1), h = (u128)(heads - 1);
                const Span ins[] = {span(q, 2 * (t * qt + h * qh + c.dim)), span(c.k, cache_bytes(c, c.k_stride)),
                                    span(c.v, cache_bytes(c, c.v_stride)),
                                    span(table, 4 * ((u128)(requests - 1) * stride + width)),
                                    span(start, ((u128)requests + 1) * 4), span(kv, (u128)requests * 4)};
                const Span outs[] = {span(out, (type == 0 ? 4 : 2) * (t * ot + h * oh + c.dim)), span(work, (u128)bytes)};
                apart(outs, 2, ins, 6, "attn buffers", i);
            }
            const int64_t dim = size_of(r, 128);
            require((gemv_paged_attn_workspace(dim) > 0) == (dim == 64 || dim == 128 || dim == 256), "workspace", i);
        }
    }
    std::printf("ok %ld iterations, accepted %ld %ld %ld\n", n, accepted[0], accepted[1], accepted[2]);
    return accepted[0] > 0 && accepted[1] > 0 && accepted[2] > 0 ? 0 : 1;
}

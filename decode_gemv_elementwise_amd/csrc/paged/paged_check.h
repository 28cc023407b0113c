// Host-side checks that the paged operators share: spans and their overlap, strides,
// alignment.  No HIP call and no dereference of a device pointer.
#pragma once

#include <cstdint>

#include "paged_internal.h"

namespace gemv {
namespace {

[[maybe_unused]] constexpr int64_t kInt = INT32_MAX;

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
[[maybe_unused]] bool any_overlap(const Span *outs, int nouts, const Span *ins, int nins)
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

[[maybe_unused]] bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

[[maybe_unused]] bool is_type(int t) { return t == GEMV_W_F32 || t == GEMV_W_F16 || t == GEMV_W_BF16; }

[[maybe_unused]] int64_t type_size(int t) { return t == GEMV_W_F32 ? 4 : 2; }

// Elements to bytes; a product past 64 bits is the whole address space.
uint64_t bytes_of(uint64_t elements, int64_t size)
{
    return elements > UINT64_MAX / (uint64_t)size ? UINT64_MAX : elements * (uint64_t)size;
}

// Bytes from the first row's start to the last row's end.  Strides and extents
// that reach here are below 2^31 each.
[[maybe_unused]] uint64_t strided_bytes(int64_t rows, int64_t stride, int64_t row, int64_t size)
{
    return rows == 0 ? 0 : bytes_of((uint64_t)(rows - 1) * (uint64_t)stride + (uint64_t)row, size);
}

// The strides (n up to 4) nest without two elements meeting: taken from the
// smallest up, each is at least what those below it span.
[[maybe_unused]] bool strides_nest(const int64_t *stride, const int64_t *extent, int n, int64_t row)
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

} // namespace
} // namespace gemv

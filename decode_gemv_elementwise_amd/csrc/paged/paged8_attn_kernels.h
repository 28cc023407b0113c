// gemv_paged8_attn's kernels of one head width.  Each width is a translation unit of its
// own, so that they compile side by side.
#pragma once

#include "paged8_attn_few.h"
#include "paged8_attn_many.h"

namespace gemv {
namespace {

template <int CODE, bool BF, int D, bool F32OUT> const void *kernel_of(bool runs, bool many)
{
    if (many)
        return runs ? reinterpret_cast<const void *>(&paged8_many_kernel<CODE, BF, D, F32OUT, true>)
                    : reinterpret_cast<const void *>(&paged8_many_kernel<CODE, BF, D, F32OUT, false>);
    return runs ? reinterpret_cast<const void *>(&paged8_few_kernel<CODE, BF, D, F32OUT, true>)
                : reinterpret_cast<const void *>(&paged8_few_kernel<CODE, BF, D, F32OUT, false>);
}

template <int CODE, int D> const void *kernel_of(bool bf, bool f32out, bool runs, bool many)
{
    if (bf)
        return f32out ? kernel_of<CODE, true, D, true>(runs, many) : kernel_of<CODE, true, D, false>(runs, many);
    return f32out ? kernel_of<CODE, false, D, true>(runs, many) : kernel_of<CODE, false, D, false>(runs, many);
}

template <int D> const void *kernel_of(int code, bool bf, bool f32out, bool runs, bool many)
{
    return code == GEMV_KV_INT8 ? kernel_of<GEMV_KV_INT8, D>(bf, f32out, runs, many)
                                : kernel_of<GEMV_KV_E4M3, D>(bf, f32out, runs, many);
}

} // namespace
} // namespace gemv

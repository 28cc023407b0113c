// gemv_paged8_attn's kernels for heads of 128 values.
#include "paged8_attn_kernels.h"

namespace gemv {

const void *paged8_attn_kernel_128(int code, bool bf, bool f32out, bool runs, bool many)
{
    return kernel_of<128>(code, bf, f32out, runs, many);
}

} // namespace gemv

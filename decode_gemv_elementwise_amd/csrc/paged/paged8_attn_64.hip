// gemv_paged8_attn's kernels for heads of 64 values.
#include "paged8_attn_kernels.h"

namespace gemv {

const void *paged8_attn_kernel_64(int code, bool bf, bool f32out, bool runs, bool many)
{
    return kernel_of<64>(code, bf, f32out, runs, many);
}

} // namespace gemv

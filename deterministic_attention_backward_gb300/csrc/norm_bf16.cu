// norm_bf16.cu -- the row norms for bf16 rows.
#include "norm_kernel.cuh"

namespace dash {
DASH_NORM_TYPE(__nv_bfloat16)
}  // namespace dash

// norm_fp16.cu -- the row norms for fp16 rows.
#include "norm_kernel.cuh"

namespace dash {
DASH_NORM_TYPE(__half)
}  // namespace dash

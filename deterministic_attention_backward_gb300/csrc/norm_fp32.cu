// norm_fp32.cu -- the row norms for fp32 rows.
#include "norm_kernel.cuh"

namespace dash {
DASH_NORM_TYPE(float)
}  // namespace dash

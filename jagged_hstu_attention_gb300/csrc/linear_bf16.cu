// The linear maps' tcgen05 kernels for bf16 rows.
#include "linear.cuh"

namespace hstu {
HSTU_LINEAR_LAUNCHES(__nv_bfloat16, bf16)
}  // namespace hstu

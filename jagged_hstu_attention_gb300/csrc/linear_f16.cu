// The linear maps' tcgen05 kernels for fp16 rows.
#include "linear.cuh"

namespace hstu {
HSTU_LINEAR_LAUNCHES(__half, f16)
}  // namespace hstu

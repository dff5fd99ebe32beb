// Paged attention kernels for bf16 rows and pages.
#include "paged_many.cuh"

namespace hstu {

cudaError_t launch_paged_bf16(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_paged_typed<__nv_bfloat16, false>(p, blocks, stream);
}

}  // namespace hstu

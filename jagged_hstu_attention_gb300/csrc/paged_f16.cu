// Paged attention kernels for fp16 rows and pages.
#include "paged_many.cuh"

namespace hstu {

cudaError_t launch_paged_f16(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_paged_typed<__half, false>(p, blocks, stream);
}

}  // namespace hstu

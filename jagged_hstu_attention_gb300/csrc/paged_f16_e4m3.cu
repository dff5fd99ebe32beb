// Paged attention kernels for fp16 rows, 8-bit pages.
#include "paged_many.cuh"

namespace hstu {

cudaError_t launch_paged_f16_e4m3(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_paged_typed<__half, true>(p, blocks, stream);
}

}  // namespace hstu

// Paged attention kernels for bf16 rows, 8-bit pages.
#include "paged_many.cuh"

namespace hstu {

cudaError_t launch_paged_bf16_e4m3(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  return launch_paged_typed<__nv_bfloat16, true>(p, blocks, stream);
}

}  // namespace hstu

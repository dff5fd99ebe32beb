// What linear.cu launches: the kernels of one type are compiled in a translation
// unit of their own.
#pragma once

#include "gemm_few.cuh"

namespace hstu {

// kEpiLinear with K-major operands (8-bit with f8).
cudaError_t launch_linear_bf16(const LinearParams& p, bool f8, cudaStream_t stream);
cudaError_t launch_linear_f16(const LinearParams& p, bool f8, cudaStream_t stream);
// The same for few rows.
cudaError_t launch_few_bf16(const FewParams& p, bool f8, cudaStream_t stream);
cudaError_t launch_few_f16(const FewParams& p, bool f8, cudaStream_t stream);
cudaError_t launch_few_dx_bf16(const FewParams& p, cudaStream_t stream);
cudaError_t launch_few_dx_f16(const FewParams& p, cudaStream_t stream);
// dx = g w: A K-major, B MN-major.
cudaError_t launch_linear_dx_bf16(const LinearParams& p, cudaStream_t stream);
cudaError_t launch_linear_dx_f16(const LinearParams& p, cudaStream_t stream);
// dw = g^T x: both MN-major; fp32 parts where k_splits > 1.
cudaError_t launch_linear_dw_bf16(const LinearParams& p, cudaStream_t stream);
cudaError_t launch_linear_dw_f16(const LinearParams& p, cudaStream_t stream);

template <typename T, bool F8, bool A_MN, bool B_MN, int EPI, int TN = kTileN>
cudaError_t launch_pair_gemm(const LinearParams& p, cudaStream_t stream) {
  const int smem = static_cast<int>(sizeof(GemmSmem2<TN>)) + 1024;
  static std::atomic<uint64_t> configured{0};
  auto kernel = pair_gemm_kernel<T, F8, A_MN, B_MN, EPI, TN>;
  cudaError_t e = ensure_smem_limit(kernel, smem, configured);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int64_t tiles = int64_t{(p.M + kTileM - 1) / kTileM} * ((p.N + TN - 1) / TN) * p.k_splits;
  const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
  return launch_chained(kernel, dim3(static_cast<unsigned>(2 * pairs)), kGemmThreads2, smem, stream, p);
}
template <typename T, bool F8, bool B_MN, int EPI>
cudaError_t launch_rows_gemm(const LinearParams& p, cudaStream_t stream) {
  return p.narrow ? launch_pair_gemm<T, F8, false, B_MN, EPI, kTileN / 2>(p, stream)
                  : launch_pair_gemm<T, F8, false, B_MN, EPI>(p, stream);
}

// Instantiates the launches of one type.
#define HSTU_LINEAR_LAUNCHES(T, SUFFIX)                                                                     \
  cudaError_t launch_linear_##SUFFIX(const LinearParams& p, bool f8, cudaStream_t stream) {                 \
    return f8 ? launch_rows_gemm<T, true, false, kEpiLinear>(p, stream)                                     \
              : launch_rows_gemm<T, false, false, kEpiLinear>(p, stream);                                   \
  }                                                                                                         \
  cudaError_t launch_few_##SUFFIX(const FewParams& p, bool f8, cudaStream_t stream) {                       \
    return f8 ? launch_few<T, true, false>(p, stream) : launch_few<T, false, false>(p, stream);             \
  }                                                                                                         \
  cudaError_t launch_few_dx_##SUFFIX(const FewParams& p, cudaStream_t stream) {                             \
    return launch_few<T, false, true>(p, stream);                                                           \
  }                                                                                                         \
  cudaError_t launch_linear_dx_##SUFFIX(const LinearParams& p, cudaStream_t stream) {                       \
    return launch_rows_gemm<T, false, true, kEpiPlain>(p, stream);                                          \
  }                                                                                                         \
  cudaError_t launch_linear_dw_##SUFFIX(const LinearParams& p, cudaStream_t stream) {                       \
    return p.k_splits > 1 ? launch_pair_gemm<T, false, true, true, kEpiPartial32>(p, stream)                \
                          : launch_pair_gemm<T, false, true, true, kEpiPlain>(p, stream);                   \
  }

}  // namespace hstu

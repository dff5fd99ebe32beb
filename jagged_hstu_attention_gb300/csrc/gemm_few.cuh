// The linear maps for few rows, where the weight is what there is to read: the
// product transposed, 128 outputs x up to 64 rows a CTA on tcgen05 (A = 128 rows of
// w, B = the rows of x), K split over a cluster of up to eight CTAs.
//
// A step of 64 rows has 16 tiles at 2048 outputs; with K = 512 split eight ways 128
// CTAs each fetch one 24 KB block, which is all the waiting there is. Operands come by
// 16-byte asynchronous copies written where the MMA expects them (128-byte
// swizzle), with no tensor maps to encode on the host. The CTAs' sums meet in
// distributed shared memory: each CTA adds its part of the rows over the cluster, in
// rank order, and runs their epilogue.
#pragma once

#include "gemm.cuh"

namespace hstu {

constexpr int kFewThreads = 256, kFewStages = 4, kFewOutputs = 128, kFewRows = 64;

struct FewParams {
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  const uint8_t* x_scale;
  const uint8_t* w_scale;
  void* y;
  void* z;
  int32_t* header;
  int64_t x_stride, residual_stride;  // bytes; elements
  int64_t k_bytes;                    // of a row
  int32_t M, N, act;
};

inline int64_t few_tiles(int64_t rows, int outputs, int tile_rows) {
  return (rows + tile_rows - 1) / tile_rows * ((outputs + kFewOutputs - 1) / kFewOutputs);
}

template <int NT>
struct FewSmem {
  alignas(1024) uint8_t a[kFewStages][kFewOutputs * 128];
  alignas(1024) uint8_t b[kFewStages][NT * 128];
  alignas(8) uint64_t done[kFewStages];
  uint32_t tmem_base;
  int abort_flag;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ float4 lds_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
template <bool F8>
__device__ __forceinline__ void umma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (!F8) return umma_ss(d, a, b, idesc, accumulate);
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Copies 128 bytes of rows [row0, row0 + ROWS) of a matrix of `rows` rows, from byte
// 128 kb on; what lies outside it becomes zeros.
template <int ROWS>
__device__ __forceinline__ void copy_block(uint32_t dst, const uint8_t* src, int64_t stride, int row0, int rows,
                                           int64_t k_bytes, int kb) {
#pragma unroll
  for (int i = threadIdx.x; i < ROWS * 8; i += kFewThreads) {
    const int r = i >> 3, c = i & 7;
    const int64_t byte = int64_t{128} * kb + 16 * c;
    const bool valid = row0 + r < rows && byte < k_bytes;
    copy16(dst + r * 128 + ((c ^ (r & 7)) << 4), valid ? src + (row0 + r) * stride + byte : src, valid);
  }
}

template <typename T, bool F8, int NT>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  FewSmem<NT>& s = *reinterpret_cast<FewSmem<NT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kColumns = NT < 32 ? 32 : NT;  // of TMEM
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;  // the cluster lies along x
  const int n0 = blockIdx.y * kFewOutputs, m0 = blockIdx.z * NT;
  const int nk = static_cast<int>((p.k_bytes + 127) / 128);
  const int kb0 = static_cast<int>(static_cast<int64_t>(nk) * rank / split);
  const int blocks = static_cast<int>(static_cast<int64_t>(nk) * (rank + 1) / split) - kb0;  // one at least
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kFewStages; ++i) mbar_init(smem_u32(&s.done[i]), 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&s.tmem_base), kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tacc = s.tmem_base;
  chain();

  const uint8_t *x = static_cast<const uint8_t*>(p.x), *w = static_cast<const uint8_t*>(p.w);
  auto load = [&](int j) {
    if (j < blocks) {
      copy_block<kFewOutputs>(smem_u32(s.a[j % kFewStages]), w, p.k_bytes, n0, p.N, p.k_bytes, kb0 + j);
      copy_block<NT>(smem_u32(s.b[j % kFewStages]), x, p.x_stride, m0, p.M, p.k_bytes, kb0 + j);
    }
    copy_commit();
  };
  for (int j = 0; j < kFewStages - 1; ++j) load(j);
  constexpr uint32_t idesc = idesc_f16kind(kFewOutputs, NT, false, false, F8 ? 0u : Elem<T>::kUmma);
  bool ok = true;
  for (int j = 0; j < blocks; ++j) {
    copy_wait<kFewStages - 2>();
    fence_async_smem();
    ok = __syncthreads_and(ok);  // block j has arrived; all agree whether to go on
    if (!ok) break;
    if (warp == 0 && elect_one_sync()) {
      const uint32_t a = smem_u32(s.a[j % kFewStages]), b = smem_u32(s.b[j % kFewStages]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_one<F8>(tacc, block_desc<false>(a, kk), block_desc<false>(b, kk), idesc, j > 0 || kk > 0 ? 1u : 0u);
      umma_commit(smem_u32(&s.done[j % kFewStages]));
    }
    __syncwarp();
    // The block before has been multiplied: its stage takes the next one to come.
    if (j > 0) ok = mbar_wait(smem_u32(&s.done[(j - 1) % kFewStages]), ((j - 1) / kFewStages) & 1, &s.abort_flag);
    if (ok) load(j + kFewStages - 1);
  }
  copy_wait<0>();
  if (ok) ok = mbar_wait(smem_u32(&s.done[(blocks - 1) % kFewStages]), ((blocks - 1) / kFewStages) & 1, &s.abort_flag);
  ok = __syncthreads_and(ok);
  tc_fence_after();
  // The CTA's sums as [row][output], over the operands, which nothing reads any more.
  const uint32_t part = smem_u32(s.a[0]);
  static_assert(NT * kFewOutputs * 4 <= sizeof(s.a), "sums over the operands");
  if (ok && warp < 4) {
#pragma unroll
    for (int c = 0; c < NT; c += 32) {
      uint32_t a[32];
      tmem_ld32(tacc + (static_cast<uint32_t>(warp * 32) << 16) + c, a);
      tmem_ld_wait(a);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (c + e < NT)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(part + ((c + e) * kFewOutputs + warp * 32 + lane) * 4), "r"(a[e])
                       : "memory");
    }
  }
  // Rows [rank NT / split, (rank + 1) NT / split) are this CTA's, four outputs a thread.
  const int r0 = rank * NT / split, r1 = (rank + 1) * NT / split;
  const int col = n0 + lane * 4;
  uint2 bias = make_uint2(0, 0);
  uint32_t col_scale = 0;
  if (col < p.N) {
    if (p.bias) bias = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.bias) + col);
    if (F8) col_scale = *reinterpret_cast<const uint32_t*>(p.w_scale + col);
  }
  cluster_sync();  // all sums are in place
  for (int r = r0 + warp; r < r1; r += kFewThreads / 32) {
    const int row = m0 + r;
    if (!ok || row >= p.M || col >= p.N) continue;
    uint2 res = make_uint2(0, 0);
    if (p.residual) res = *reinterpret_cast<const uint2*>(static_cast<const T*>(p.residual) + row * p.residual_stride + col);
    const float row_scale = F8 ? scale_value(p.x_scale[row]) : 1.0f;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const uint32_t mine = part + (r * kFewOutputs + lane * 4) * 4;
#pragma unroll 8
    for (int c = 0; c < split; ++c) {
      const float4 v = lds_cluster(in_cta(mine, c));
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    uint64_t v[2] = {pair_of(sum.x, sum.y), pair_of(sum.z, sum.w)};
    const uint32_t bw[2] = {bias.x, bias.y}, rw[2] = {res.x, res.y};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (F8) {
        const uint32_t b = col_scale >> (16 * e);
        v[e] = pair_mul(pair_mul(v[e], pair_of(row_scale, row_scale)),
                        pair_of(scale_value(b & 0xffu), scale_value((b >> 8) & 0xffu)));
      }
      v[e] = pair_add(v[e], unpack_pair<T>(bw[e]));
    }
    const int64_t at = static_cast<int64_t>(row) * p.N + col;
    if (p.z) *reinterpret_cast<uint2*>(static_cast<T*>(p.z) + at) = make_uint2(pack_pair<T>(v[0]), pack_pair<T>(v[1]));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (p.act == HSTU_ACT_SILU) v[e] = activate2<HSTU_ACT_SILU>(v[e]);
      if (p.act == HSTU_ACT_GELU) v[e] = activate2<HSTU_ACT_GELU>(v[e]);
      if (p.act == HSTU_ACT_RELU) v[e] = activate2<HSTU_ACT_RELU>(v[e]);
      if (p.residual) v[e] = pair_add(v[e], unpack_pair<T>(rw[e]));
    }
    *reinterpret_cast<uint2*>(static_cast<T*>(p.y) + at) = make_uint2(pack_pair<T>(v[0]), pack_pair<T>(v[1]));
  }
  tc_fence_before();
  cluster_sync();  // nobody leaves while another CTA reads its sums
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tacc, kColumns);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.header) atomicOr(p.header + kHdrErr, kErrTimeout);
}

template <typename T, bool F8, int NT>
cudaError_t launch_few_rows(const FewParams& p, cudaStream_t stream) {
  const int smem = static_cast<int>(sizeof(FewSmem<NT>)) + 1024;
  static std::atomic<uint64_t> configured{0};
  auto kernel = few_rows_kernel<T, F8, NT>;
  const cudaError_t e = ensure_smem_limit(kernel, smem, configured);
  if (e != cudaSuccess) return e;
  // K is split until there are as many CTAs as SMs, eight ways at most; twice as many
  // where a CTA still has four blocks then (64 x 2048 x 2048: 7.7 us so, 8.3 us split
  // four ways; 64 x 512 x 2048: 5.8 and 5.4).
  const int64_t nk = (p.k_bytes + 127) / 128, tiles = few_tiles(p.M, p.N, NT);
  int split = 1;
  while (split < 8 && 2 * split <= nk && tiles * split * 2 <= (nk / (2 * split) >= 4 ? 2 * 152 : 152)) split *= 2;
  cudaLaunchAttribute attrs[2]{};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim = {static_cast<unsigned>(split), 1, 1};
  cudaLaunchConfig_t config{};
  config.gridDim = dim3(split, (p.N + kFewOutputs - 1) / kFewOutputs, (p.M + NT - 1) / NT);
  config.blockDim = dim3(kFewThreads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = attrs;
  config.numAttrs = 2;
  return cudaLaunchKernelEx(&config, kernel, p);
}
// Fewer rows a tile, whose sums take less time to meet, where all tiles, split four
// ways, still fit the SMs (64 x 512 x 2048: 5.4 us with tiles of 32 rows, 6.1 us with
// 64; 64 x 4096 x 4096: 13.9 and 11.9).
template <typename T, bool F8>
cudaError_t launch_few(const FewParams& p, cudaStream_t stream) {
  if (p.M <= 16 || 4 * few_tiles(p.M, p.N, 16) <= 152) return launch_few_rows<T, F8, 16>(p, stream);
  if (p.M <= 32 || 4 * few_tiles(p.M, p.N, 32) <= 152) return launch_few_rows<T, F8, 32>(p, stream);
  return launch_few_rows<T, F8, 64>(p, stream);
}

}  // namespace hstu

// The linear maps for few rows, where the weight is what there is to read: the
// product transposed, 128 outputs x up to 64 rows a CTA on tcgen05 (A = 128 rows of
// w, B = the rows of x), K split over a cluster of up to eight CTAs.
//
// A step of 64 rows has 16 tiles at 2048 outputs; with K = 512 split eight ways 128
// CTAs each fetch one 24 KB block, which is all the waiting there is. Operands come by
// 16-byte asynchronous copies written where the MMA expects them (128-byte
// swizzle), with no tensor maps to encode on the host. The CTAs' sums meet in
// distributed shared memory: each CTA writes its sums of a part of the rows to the CTA
// that owns the part, which adds them in rank order and runs the epilogue. (Read from
// where they were computed instead, with a second barrier before anyone may leave: 64
// rows, 512 x 2048, in 5.4 us.)
#pragma once

#include "gemm.cuh"

namespace hstu {

constexpr int kFewThreads = 256, kFewOutputs = 128, kFewRows = 64;
constexpr int kFewMostStages = 5;
template <int NT>
constexpr int kFewStageBytes = (kFewOutputs + NT) * 128;
template <int NT>
constexpr int kFewMeetBytes = NT * kFewOutputs * 4;
// K blocks in shared memory, where a CTA has as many: two CTAs share an SM up to 64
// rows. (A block takes a CTA about 0.55 us however many are on their way, so that two
// CTAs with three stages beat one with seven: 64 x 4096 x 4096 11.9 and 15.2 us.)
template <int NT>
constexpr int kFewStages = NT == 16 ? 5 : NT == 32 ? 4 : 3;

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
  int32_t stages;
  bool give_up;  // a test's: the wait for the last products gives up at once, with MMAs in flight
};

inline int64_t few_tiles(int64_t rows, int outputs, int tile_rows) {
  return (rows + tile_rows - 1) / tile_rows * ((outputs + kFewOutputs - 1) / kFewOutputs);
}

struct FewSmem {  // the stages and the sums of others lie behind
  uint64_t done[kFewMostStages], drain;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(FewSmem) <= 256, "the space in front of the stages");

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `n` of the groups committed last are on their way.
__device__ __forceinline__ void copy_wait_all_but(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}
// The halves of a cluster barrier; the arrival orders nothing.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void sts_cluster(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
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

// The same of a matrix whose columns are the outputs (MN-major): columns [col0, col0 + 128) of
// rows [64 kb, 64 kb + 64), as [64-column group][row][128 bytes].
__device__ __forceinline__ void copy_block_mn(uint32_t dst, const uint8_t* src, int col0, int cols, int64_t rows, int kb) {
#pragma unroll
  for (int i = threadIdx.x; i < 64 * 16; i += kFewThreads) {
    const int r = i >> 4, c = i & 15;
    const int64_t row = int64_t{64} * kb + r;
    const bool valid = row < rows && col0 + 8 * c < cols;
    copy16(dst + (c >> 3) * 64 * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4),
           valid ? src + (row * cols + col0 + 8 * c) * 2 : src, valid);
  }
}

// W_MN: w is (K, N), its columns the outputs (the gradient of the rows).
template <typename T, bool F8, bool W_MN, int NT>
__global__ void __launch_bounds__(kFewThreads) few_rows_kernel(const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  cluster_arrive();  // this CTA has started: what the others wait for before they write here
  // [stages: A 16 KB, B], sums [CTA][pair of own rows][output], barriers
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float2* meet = reinterpret_cast<float2*>(base + p.stages * kFewStageBytes<NT>);
  FewSmem& s = *reinterpret_cast<FewSmem*>(reinterpret_cast<uint8_t*>(meet) + kFewMeetBytes<NT>);
  constexpr int kColumns = NT < 32 ? 32 : NT;  // of TMEM
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = gridDim.x, rank = blockIdx.x;  // the cluster lies along x
  const int n0 = blockIdx.y * kFewOutputs, m0 = blockIdx.z * NT;
  const int nk = static_cast<int>((p.k_bytes + 127) / 128);
  const int kb0 = static_cast<int>(static_cast<int64_t>(nk) * rank / split);
  const int blocks = static_cast<int>(static_cast<int64_t>(nk) * (rank + 1) / split) - kb0;  // one at least
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < p.stages; ++i) mbar_init(smem_u32(&s.done[i]), 1);
    mbar_init(smem_u32(&s.drain), 1);
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
  const uint32_t ring = smem_u32(base);
  auto stage_of = [&](int st) { return ring + st * kFewStageBytes<NT>; };
  int loaded = 0, load_st = 0;  // blocks on their way; the stage of the next
  auto load = [&] {
    if (loaded < blocks) {
      const uint32_t a = stage_of(load_st);
      if (W_MN) copy_block_mn(a, w, n0, p.N, p.k_bytes / 2, kb0 + loaded);
      else copy_block<kFewOutputs>(a, w, p.k_bytes, n0, p.N, p.k_bytes, kb0 + loaded);
      copy_block<NT>(a + kFewOutputs * 128, x, p.x_stride, m0, p.M, p.k_bytes, kb0 + loaded);
    }
    ++loaded;
    if (++load_st == p.stages) load_st = 0;
    copy_commit();
  };
  for (int j = 0; j < p.stages - 1; ++j) load();
  constexpr uint32_t idesc = idesc_f16kind(kFewOutputs, NT, W_MN, false, F8 ? 0u : Elem<T>::kUmma);
  bool ok = true;
  int st = 0, phase = 0, before = 0, before_phase = 0;  // of this block and the one before
  for (int j = 0; j < blocks; ++j) {
    copy_wait_all_but(p.stages - 2);
    fence_async_smem();
    ok = __syncthreads_and(ok);  // block j has arrived; all agree whether to go on
    if (!ok) break;
    if (warp == 0 && elect_one_sync()) {
      const uint32_t a = stage_of(st), b = a + kFewOutputs * 128;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_one<F8>(tacc, block_desc<W_MN>(a, kk), block_desc<false>(b, kk), idesc, j > 0 || kk > 0 ? 1u : 0u);
      umma_commit(smem_u32(&s.done[st]));
    }
    __syncwarp();
    // The block before has been multiplied: its stage takes the next one to come.
    if (j > 0) ok = mbar_wait(smem_u32(&s.done[before]), before_phase, &s.abort_flag);
    if (ok) load();
    before = st;
    before_phase = phase;
    if (++st == p.stages) st = 0, phase ^= 1;
  }
  copy_wait_all_but(0);
  if (ok) ok = !p.give_up && mbar_wait(smem_u32(&s.done[before]), before_phase, &s.abort_flag);
  ok = __syncthreads_and(ok);
  if (!ok) {  // MMAs may be on their way still
    if (warp == 0 && elect_one_sync()) {
      s.abort_flag = 1;
      umma_commit(smem_u32(&s.drain));
      mbar_wait_drain(smem_u32(&s.drain), 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  // Rows [c own, (c + 1) own) of the tile are CTA c's: sums of pairs of rows, an output
  // a lane; warps 4 to 7 take the second half of the columns.
  const int own = NT / split;
  cluster_wait();  // all CTAs have started
  if (ok) {
    constexpr int kHalf = NT / 2;
    const int c0 = warp < 4 ? 0 : kHalf, output = (warp & 3) * 32 + lane;
    uint32_t a[32];
    tmem_ld32(tacc + (static_cast<uint32_t>((warp & 3) * 32) << 16) + (NT < 64 ? 0 : c0), a);
    tmem_ld_wait(a);
#pragma unroll
    for (int e = 0; e < kHalf; e += 2) {
      const int row = c0 + e, at = rank * own + row % own;
      const bool second = NT < 64 && warp >= 4;  // the columns of both halves were read
      sts_cluster(in_cta(smem_u32(&meet[at / 2 * kFewOutputs + output]), row / own), second ? a[(kHalf + e) & 31] : a[e],
                  second ? a[(kHalf + e + 1) & 31] : a[e + 1]);
    }
  }
  const int output = threadIdx.x % kFewOutputs, col = n0 + output;
  tc_fence_before();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // What the rows and columns need is read while the sums meet: behind the arrival, which
  // would wait for it (0.2 us), and as it lies in memory.
  uint16_t bias_bits = 0, next_res[2] = {0, 0};
  uint8_t col_byte = 0, next_byte[2] = {0, 0};
  if (col < p.N) {
    if (p.bias) bias_bits = static_cast<const uint16_t*>(p.bias)[col];
    if (F8) col_byte = p.w_scale[col];
  }
  auto read_rows = [&](int j) {
    const int row = m0 + rank * own + 2 * j;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (j >= own / 2 || row + e >= p.M || col >= p.N) continue;
      if (p.residual) next_res[e] = static_cast<const uint16_t*>(p.residual)[(row + e) * p.residual_stride + col];
      if (F8) next_byte[e] = p.x_scale[row + e];
    }
  };
  constexpr int kRowStep = kFewThreads / kFewOutputs;
  read_rows(threadIdx.x / kFewOutputs);
  cluster_wait();  // all sums are in place
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tacc, kColumns);
  }
  const uint64_t bias = unpack_pair<T>(bias_bits * 0x10001u);
  for (int j = threadIdx.x / kFewOutputs; j < own / 2; j += kRowStep) {
    const int row = m0 + rank * own + 2 * j;
    const uint32_t res = next_res[0] | static_cast<uint32_t>(next_res[1]) << 16;
    const uint8_t row_byte[2] = {next_byte[0], next_byte[1]};
    read_rows(j + kRowStep);
    if (!ok || row >= p.M || col >= p.N) continue;
    const bool second = row + 1 < p.M;
    const int64_t at = static_cast<int64_t>(row) * p.N + col;
    uint64_t v = pair_of(0.0f, 0.0f);
#pragma unroll 8
    for (int c = 0; c < split; ++c) {
      const float2 f = meet[(c * own / 2 + j) * kFewOutputs + output];
      v = pair_add(v, pair_of(f.x, f.y));
    }
    if (F8)  // by w's scale first, as in the pair kernel
      v = pair_mul(pair_mul(v, pair_of(scale_value(col_byte), scale_value(col_byte))),
                   pair_of(scale_value(row_byte[0]), scale_value(row_byte[1])));
    v = pair_add(v, bias);
    auto store = [&](void* base, uint64_t values) {
      const uint32_t w = pack_pair<T>(values);
      uint16_t* to = static_cast<uint16_t*>(base) + at;
      to[0] = static_cast<uint16_t>(w);
      if (second) to[p.N] = static_cast<uint16_t>(w >> 16);
    };
    if (p.z) store(p.z, v);
    if (p.act == HSTU_ACT_SILU) v = activate2<HSTU_ACT_SILU>(v);
    if (p.act == HSTU_ACT_GELU) v = activate2<HSTU_ACT_GELU>(v);
    if (p.act == HSTU_ACT_RELU) v = activate2<HSTU_ACT_RELU>(v);
    if (p.residual) v = pair_add(v, unpack_pair<T>(res));
    store(p.y, v);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.header) atomicOr(p.header + kHdrErr, kErrTimeout);
}

// Rows of a tile, and K's splits over a cluster, eight at most: until there is a CTA for
// each SM, or two where a CTA keeps four blocks. The cost is a model of the measured time
// in units of 10 ns: launch, meeting sums, blocks one after the other, slower where two
// CTAs share an SM. (64 rows: 512 x 2048 takes 5.1 us with tiles of 32 rows, 6.0 us with 64;
// 4096 x 4096 13.7 and 11.8. Tiles of 128 rows gained nothing: 384 x 8192 x 1024 26.1 us, 26.0 with 64.)
struct FewPlan {
  int rows_tile = 0, split = 1;
  int64_t cost = INT64_MAX;
};
inline FewPlan few_plan(int64_t rows, int outputs, int64_t k_bytes) {
  FewPlan best;
  const int64_t nk = (k_bytes + 127) / 128;
  for (int nt = 16; nt <= kFewRows; nt *= 2) {
    const int64_t tiles = few_tiles(rows, outputs, nt);
    int split = 1;
    while (split < 8 && 2 * split <= nk && tiles * split * 2 <= (nk / (2 * split) >= 4 ? 304 : 152)) split *= 2;
    const int64_t ctas = tiles * split, blocks = (nk + split - 1) / split, waves = (ctas + 303) / 304;
    const int64_t block = (nt < 64 ? 55 : 70) * (ctas > 152 ? 13 : 10) / 10;
    const int64_t cost = 330 + waves * ((nt <= 32 ? 3 * nt - 15 : 185) + blocks * block);
    if (cost < best.cost) best = FewPlan{nt, split, cost};
  }
  return best;
}

template <typename T, bool F8, bool W_MN, int NT>
cudaError_t launch_few_rows(const FewParams& given, int split, cudaStream_t stream) {
  FewParams p = given;
  const int64_t nk = (p.k_bytes + 127) / 128, blocks = (nk + split - 1) / split;
  p.stages = static_cast<int>(blocks < 2 ? 2 : (blocks < kFewStages<NT> ? blocks : kFewStages<NT>));
  const int smem = p.stages * kFewStageBytes<NT> + kFewMeetBytes<NT> + 256 + 1024;
  static std::atomic<uint64_t> configured{0};
  auto kernel = few_rows_kernel<T, F8, W_MN, NT>;
  const cudaError_t e =
      ensure_smem_limit(kernel, kFewStages<NT> * kFewStageBytes<NT> + kFewMeetBytes<NT> + 256 + 1024, configured);
  if (e != cudaSuccess) return e;
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
template <typename T, bool F8, bool W_MN>
cudaError_t launch_few(const FewParams& p, cudaStream_t stream) {
  const FewPlan plan = few_plan(p.M, p.N, p.k_bytes);
  switch (plan.rows_tile) {
    case 16: return launch_few_rows<T, F8, W_MN, 16>(p, plan.split, stream);
    case 32: return launch_few_rows<T, F8, W_MN, 32>(p, plan.split, stream);
    default: return launch_few_rows<T, F8, W_MN, 64>(p, plan.split, stream);
  }
}

}  // namespace hstu

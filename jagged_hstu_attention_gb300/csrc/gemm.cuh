// Matrix products on tcgen05 for the layer's linear maps: C[M x N] = A[M x K] B[N x K]^T
// with fp32 accumulation in TMEM, 16-bit or 8-bit (e4m3) operands.
//
// Two CTAs of a cluster work on one 256 x 256 tile (cta_group::2): each holds 128 rows
// of A and 128 of B, the leader's MMAs (M = 256, N = 256) read both, and each CTA's
// TMEM gets its own 128 rows of the result. A CTA so loads 256 operand rows for each K
// block instead of the 384 that a 128 x 256 tile of its own takes. Persistent: a pair
// takes tiles in turn, N fastest, so that pairs running together share A's rows and
// B stays in L2. 128-byte deep K blocks (64 16-bit or 128 8-bit values) flow through
// a ring of five TMA stages that runs on across tiles; two 256-column accumulators, so
// that eight epilogue warps read one out while the next is computed.
//
// An operand is K-major when K runs along its tensor's rows, MN-major when K runs
// down its columns (boxes of 64 columns x 64 rows, 16-bit only).
#pragma once

#include "../../include/hstu_attn.h"
#include "cache.cuh"
#include "internal.h"

namespace hstu {

constexpr int kTileM = 256, kTileN = 256;        // of a pair
constexpr int kStages = 5;
constexpr int kStageOperand = 128 * 128;         // bytes of A and of B in a stage of one CTA
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads2 = (kEpiWarps + 2) * 32;  // epilogue, TMA producer, MMA issuer

// Epilogues.
constexpr int kEpiLinear = 0;    // y = act(acc scales + bias) + residual, z before act
constexpr int kEpiPlain = 1;     // y = acc
constexpr int kEpiPartial32 = 2; // part[split] = acc in fp32 (split K)

struct LinearParams {
  CUtensorMap tm_a, tm_b;
  CUtensorMap tm_y, tm_z, tm_r;  // boxes of 64 columns x 32 rows
  const void* bias;              // nullable, (N)
  const uint8_t* a_scale;        // 8-bit operands: exponent bytes of A's and B's rows
  const uint8_t* b_scale;
  float* part;                   // kEpiPartial32: (k_splits, M, N)
  int32_t* header;               // nullable error word
  uint64_t handoff_limit_ns;     // of the wait for an accumulator to be read out
  int32_t M, N, K, k_splits;
  int32_t act;
  bool has_z, has_r;
};

struct GemmSmem2 {
  alignas(1024) uint8_t a[kStages][kStageOperand];
  alignas(1024) uint8_t b[kStages][kStageOperand];
  // Of each epilogue warp, 32 rows x 64 columns in the 128-byte swizzle of the maps:
  // y on its way out; z on its way out, or residual rows on their way in.
  alignas(1024) uint8_t stage_y[kEpiWarps][32 * 128];
  alignas(1024) uint8_t stage_zr[kEpiWarps][32 * 128];
  alignas(8) uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drain, res[kEpiWarps];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(GemmSmem2) + 1024 <= 232448, "over the shared memory of a CTA");

// ---------------------------------------------------------- cluster helpers
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// 2-D load whose bytes are counted by a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_load_own(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store_box(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------------ pair of CTAs
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
template <bool F8>
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  if (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives once on the barrier at this offset in both CTAs when every tcgen05
// operation that this thread issued has completed.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Loads 128 rows (K-major) or columns (MN-major) of an operand, one K block deep.
template <bool MN, int KB>
__device__ __forceinline__ void load_block(uint32_t dst, const CUtensorMap* map, uint32_t bar, int mn, int kb) {
  if (MN) {  // [64-column group][K row][128 bytes]
    tma_load_pair(dst, map, bar, mn, kb * KB);
    tma_load_pair(dst + 64 * 128, map, bar, mn + 64, kb * KB);
  } else {
    tma_load_pair(dst, map, bar, kb * KB, mn);
  }
}
template <bool MN>
__device__ __forceinline__ uint64_t block_desc(uint32_t base, int kk) {
  if (MN) return sdesc_sw128(base + kk * 16 * 128, 64 * 128, 1024);
  return sdesc_sw128(base + kk * 32, 16, 1024);
}

// ------------------------------------------------------------- activations
// x / (1 + exp(-u)): u = x is SiLU; u = 2 sqrt(2 / pi) (x + 0.044715 x^3) the tanh form of GELU.
__device__ __forceinline__ float gated(float x, float u) { return __fdividef(x, 1.0f + __expf(-u)); }
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;  // 2 sqrt(2 / pi)
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == HSTU_ACT_SILU) return gated(x, x);
  if (ACT == HSTU_ACT_GELU) return gated(x, kGeluA * x * fmaf(kGeluB * x, x, 1.0f));
  if (ACT == HSTU_ACT_RELU) return x > 0.0f ? x : (x != x ? x : 0.0f);
  return x;
}
template <int ACT>
__device__ __forceinline__ void activate_all(float (&v)[64]) {
#pragma unroll
  for (int e = 0; e < 64; ++e) v[e] = activate<ACT>(v[e]);
}

template <typename T, bool F8, bool A_MN, bool B_MN, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads2, 1)
    pair_gemm_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  GemmSmem2& s = *reinterpret_cast<GemmSmem2*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int KB = F8 ? 128 : 64;  // K values of a block
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tm = (p.M + kTileM - 1) / kTileM, tn = (p.N + kTileN - 1) / kTileN;
  const int n_tiles = tm * tn * p.k_splits;
  const int nk = (p.K + KB - 1) / KB, per = (nk + p.k_splits - 1) / p.k_splits;
  // Tile t: K split t / (tm tn), then m tile, then n tile. Its K blocks are [kb0, kb1).
  auto tile_of = [&](int t, int& m0, int& n0, int& split, int& kb0, int& kb1) {
    split = t / (tm * tn);
    const int rem = t - split * tm * tn;
    m0 = (rem / tn) * kTileM;
    n0 = (rem % tn) * kTileN;
    kb0 = min(split * per, nk);
    kb1 = min(kb0 + per, nk);
  };
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), 2 * kEpiWarps);  // of both CTAs
    }
    mbar_init(smem_u32(&s.drain), 1);
    for (int i = 0; i < kEpiWarps; ++i) mbar_init(smem_u32(&s.res[i]), 1);
    fence_mbar_init();
  }
  if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(smem_u32(&s.tmem_base), 2 * kTileN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are set up
  tc_fence_after();
  const uint32_t tbase = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;
  const uint32_t peer_abort = in_cta(smem_u32(&s.abort_flag), rank ^ 1u);
  chain();  // from here on the kernel reads what earlier ones wrote

  if (warp == kEpiWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&p.tm_a);
      tma_prefetch_map(&p.tm_b);
      int last[kStages];
      for (int st = 0; st < kStages; ++st) last[st] = -1;
      int g = 0;
      bool ok = true;
      for (int t = pair; ok && t < n_tiles; t += pairs) {
        int m0, n0, split, kb0, kb1;
        tile_of(t, m0, n0, split, kb0, kb1);
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
          const int st = g % kStages, use = g / kStages;
          if (use > 0 && !mbar_wait(smem_u32(&s.empty[st]), (use - 1) & 1, abort_flag)) {
            store_cluster(peer_abort, 1);
            ok = false;
            break;
          }
          // The leader's barrier counts the bytes of both CTAs.
          if (rank == 0) mbar_expect_tx(smem_u32(&s.full[st]), 4 * kStageOperand);
          const uint32_t bar = in_cta(smem_u32(&s.full[st]), 0);
          load_block<A_MN, KB>(smem_u32(s.a[st]), &p.tm_a, bar, m0 + 128 * rank, kb);
          load_block<B_MN, KB>(smem_u32(s.b[st]), &p.tm_b, bar, n0 + 128 * rank, kb);
          last[st] = use;
        }
      }
      // Never leave with a copy in flight: the leader waits for both CTAs', and
      // the cluster barrier at the end keeps the other one.
      if (rank == 0) {
        const uint64_t t0 = globaltimer_ns();  // one limit for all: the other CTA may have stopped before a stage
        for (int st = 0; st < kStages; ++st)
          while (last[st] >= 0 && !mbar_test(smem_u32(&s.full[st]), last[st] & 1) &&
                 globaltimer_ns() - t0 < kWaitLimitNs) {
          }
      }
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one_sync()) {
      constexpr uint32_t idesc = idesc_f16kind(kTileM, kTileN, A_MN, B_MN, F8 ? 0u : Elem<T>::kUmma);
      int g = 0, i = 0;
      bool ok = true;
      for (int t = pair; ok && t < n_tiles; t += pairs, ++i) {
        int m0, n0, split, kb0, kb1;
        tile_of(t, m0, n0, split, kb0, kb1);
        const int buf = i & 1;
        // accumulator buf is free once both CTAs have read out tile i - 2
        if (i >= 2 && !mbar_wait(smem_u32(&s.acc_empty[buf]), ((i >> 1) - 1) & 1, abort_flag, p.handoff_limit_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tacc = tbase + buf * kTileN;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
          const int st = g % kStages;
          if (!mbar_wait(smem_u32(&s.full[st]), (g / kStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_pair<F8>(tacc, block_desc<A_MN>(smem_u32(s.a[st]), kk), block_desc<B_MN>(smem_u32(s.b[st]), kk), idesc,
                          (kb > kb0 || kk > 0) ? 1u : 0u);
          umma_commit_pair(smem_u32(&s.empty[st]));
        }
        if (ok) umma_commit_pair(smem_u32(&s.acc_full[buf]));
      }
      if (!ok) store_cluster(peer_abort, 1);
      umma_commit_pair(smem_u32(&s.drain));  // every MMA issued above has completed (also on abort)
      mbar_wait_drain(smem_u32(&s.drain), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // Warp w reads TMEM lanes 32 (w % 4) .. and columns 128 (w / 4) .., in two
    // chunks of 64.
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t st_y = smem_u32(s.stage_y[warp]), st_zr = smem_u32(s.stage_zr[warp]);
    const uint32_t res_bar = smem_u32(&s.res[warp]);
    const bool has_z = EPI == kEpiLinear && p.has_z, has_r = EPI == kEpiLinear && p.has_r;
    const bool ahead = has_r && !has_z;  // residual rows are loaded a chunk ahead
    // The chunk behind (t, c) that has rows and columns of the matrix.
    auto place = [&](int t, int c, int& row0, int& col) {
      int m0, n0, split, kb0, kb1;
      tile_of(t, m0, n0, split, kb0, kb1);
      row0 = m0 + 128 * static_cast<int>(rank) + quarter * 32;
      col = n0 + half * 128 + c * 64;
      return row0 < p.M && col < p.N;
    };
    auto load_residual = [&](int row0, int col) {  // lane 0
      mbar_expect_tx(res_bar, 32 * 128);
      tma_load_own(st_zr, &p.tm_r, res_bar, col, row0);
    };
    auto load_next = [&](int t, int c) {  // lane 0: the first such chunk from (t, c) on
      for (; t < n_tiles; t += pairs, c = 0)
        for (; c < 2; ++c) {
          int row0, col;
          if (place(t, c, row0, col)) {
            load_residual(row0, col);
            return;
          }
        }
    };
    if (ahead && lane == 0) load_next(pair, 0);
    uint32_t res_phase = 0;
    bool pending = false, ok = true;  // lane 0: committed stores may still read the staging buffers
    int i = 0;
    for (int t = pair; ok && t < n_tiles; t += pairs, ++i) {
      int m0, n0, split, kb0, kb1;
      tile_of(t, m0, n0, split, kb0, kb1);
      const int buf = i & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.acc_full[buf]), (i >> 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const bool none = kb1 == kb0;  // nothing accumulated: zeros
      for (int c = 0; c < 2; ++c) {
        int row0, col;
        const bool live = place(t, c, row0, col);
        const int row = row0 + lane;
        if (!live) continue;  // the same for the whole warp
        uint32_t a[32], b[32];
        const uint32_t at = tbase + buf * kTileN + lane_addr + half * 128 + c * 64;
        tmem_ld32(at, a);
        tmem_ld32(at + 32, b);
        float v[64];
        // What belongs to the columns is read while the accumulators are.
        uint4 bias[8];
        if (EPI == kEpiLinear)
#pragma unroll
          for (int q = 0; q < 8; ++q)
            bias[q] = p.bias && col + 8 * q < p.N
                          ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + col + 8 * q)
                          : make_uint4(0, 0, 0, 0);
        uint2 scale[8];
        float row_scale = 1.0f;
        if (F8) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            scale[q] = col + 8 * q < p.N ? *reinterpret_cast<const uint2*>(p.b_scale + col + 8 * q) : make_uint2(0, 0);
          if (row < p.M) row_scale = scale_value(p.a_scale[row]);
        }
        tmem_ld_wait(a);
        tmem_ld_wait(b);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          v[e] = none ? 0.0f : __uint_as_float(a[e]);
          v[32 + e] = none ? 0.0f : __uint_as_float(b[e]);
        }
        if (EPI == kEpiPartial32) {
          if (row < p.M) {
            float* dst = p.part + (static_cast<int64_t>(split) * p.M + row) * p.N + col;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (col + 8 * q < p.N)
                asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                 dst + 8 * q),
                             "f"(v[8 * q]), "f"(v[8 * q + 1]), "f"(v[8 * q + 2]), "f"(v[8 * q + 3]), "f"(v[8 * q + 4]),
                             "f"(v[8 * q + 5]), "f"(v[8 * q + 6]), "f"(v[8 * q + 7])
                             : "memory");
          }
          continue;
        }
        if (F8)
#pragma unroll
          for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t byte = ((e < 4 ? scale[q].x : scale[q].y) >> (8 * (e & 3))) & 0xffu;
              v[8 * q + e] = v[8 * q + e] * row_scale * scale_value(byte);
            }
        if (EPI == kEpiLinear)
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t w[4] = {bias[q].x, bias[q].y, bias[q].z, bias[q].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[8 * q + 2 * e] += Elem<T>::lo(w[e]);
              v[8 * q + 2 * e + 1] += Elem<T>::hi(w[e]);
            }
          }
        // The stores of the chunk before have read the staging buffers.
        if (lane == 0 && pending) store_wait_read();
        __syncwarp();
        // Row `lane`, 16-byte piece j lies at piece j ^ (lane & 7) of the row.
        const uint32_t line = static_cast<uint32_t>(lane * 128);
        if (EPI == kEpiLinear) {
          uint4 z[8];
          if (has_z)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              z[j] = make_uint4(Elem<T>::pack2(v[8 * j], v[8 * j + 1]), Elem<T>::pack2(v[8 * j + 2], v[8 * j + 3]),
                                Elem<T>::pack2(v[8 * j + 4], v[8 * j + 5]), Elem<T>::pack2(v[8 * j + 6], v[8 * j + 7]));
          switch (p.act) {
            case HSTU_ACT_SILU: activate_all<HSTU_ACT_SILU>(v); break;
            case HSTU_ACT_GELU: activate_all<HSTU_ACT_GELU>(v); break;
            case HSTU_ACT_RELU: activate_all<HSTU_ACT_RELU>(v); break;
            default: break;
          }
          if (has_r) {
            if (!ahead && lane == 0) load_residual(row0, col);
            ok = __all_sync(0xffffffffu, mbar_wait(res_bar, res_phase, abort_flag));
            if (!ok) break;
            res_phase ^= 1u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint4 r = lds128(st_zr + line + ((j ^ (lane & 7)) << 4));
              const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[8 * j + 2 * e] += Elem<T>::lo(w[e]);
                v[8 * j + 2 * e + 1] += Elem<T>::hi(w[e]);
              }
            }
            __syncwarp();
            if (ahead && lane == 0) {
              fence_async_smem();  // the buffer has been read before the next copy into it
              load_next(t, c + 1);
            }
          }
          if (has_z)
#pragma unroll
            for (int j = 0; j < 8; ++j) sts128(st_zr + line + ((j ^ (lane & 7)) << 4), z[j].x, z[j].y, z[j].z, z[j].w);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
          sts128(st_y + line + ((j ^ (lane & 7)) << 4), Elem<T>::pack2(v[8 * j], v[8 * j + 1]),
                 Elem<T>::pack2(v[8 * j + 2], v[8 * j + 3]), Elem<T>::pack2(v[8 * j + 4], v[8 * j + 5]),
                 Elem<T>::pack2(v[8 * j + 6], v[8 * j + 7]));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {  // rows and columns past the matrix are clipped by the map
          tma_store_box(&p.tm_y, st_y, col, row0);
          if (has_z) tma_store_box(&p.tm_z, st_zr, col, row0);
          store_commit();
          pending = true;
        }
      }
      tc_fence_before();
      if (ok && lane == 0) arrive_cluster(in_cta(smem_u32(&s.acc_empty[buf]), 0));
      __syncwarp();
    }
    if (!ok && lane == 0) {
      store_cluster(peer_abort, 1);
      // a residual copy in flight: the barrier's phase that has not been seen
      if (has_r) mbar_wait_drain(res_bar, res_phase);
    }
    if (lane == 0 && pending) store_wait();  // every store done before the CTA ends
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // The last arrival that the leader's MMAs send here.
  if (rank == 1 && threadIdx.x == 0) mbar_wait_drain(smem_u32(&s.drain), 0);
  __syncthreads();
  cluster_sync();  // nobody leaves while the other CTA's MMAs, copies or arrivals may reach it
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 2 * kTileN);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.header) atomicOr(p.header + kHdrErr, kErrTimeout);
}

}  // namespace hstu

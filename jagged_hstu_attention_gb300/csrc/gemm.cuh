// Matrix products on tcgen05 for the layer's linear maps: C[M x N] = A[M x K] B[N x K]^T
// with fp32 accumulation in TMEM, 16-bit or 8-bit (e4m3) operands.
//
// Two CTAs of a cluster work on one 256 x 256 tile (cta_group::2): each holds 128 rows
// of A and 128 of B, the leader's MMAs (M = 256, N = 256) read both, and each CTA's
// TMEM gets its own 128 rows of the result. A CTA so loads 256 operand rows for each K
// block instead of the 384 that a 128 x 256 tile of its own takes. Persistent: a pair
// takes tiles in turn, N fastest, so that pairs running together share A's rows and
// B stays in L2. 128-byte deep K blocks (64 16-bit or 128 8-bit values) flow through
// a ring of six TMA stages that runs on across tiles; two 256-column accumulators, so
// that sixteen epilogue warps read one out while the next is computed. Products of few
// tiles take tiles of 256 x 128, which more pairs share.
//
// An operand is K-major when K runs along its tensor's rows, MN-major when K runs
// down its columns (boxes of 64 columns x 64 rows, 16-bit only).
#pragma once

#include <type_traits>

#include "../../include/hstu_attn.h"
#include "cache.cuh"
#include "internal.h"
#include "pairs.cuh"

namespace hstu {

constexpr int kTileM = 256, kTileN = 256;  // of a pair; kTileN / 2 columns in the narrow form
// 192 KB: what a seventh stage would take serves as L1 (81920 rows, 512 x 2048, forward and
// backward 534 us with six, 556 with seven, 545 with five).
template <int TN>
constexpr int kStages = TN == kTileN ? 6 : 8;
constexpr int kStageA = 128 * 128;  // bytes of a stage of one CTA
template <int TN>
constexpr int kStageB = TN / 2 * 128;
constexpr int kEpiWarps = 16;
constexpr int kGemmThreads2 = (kEpiWarps + 2) * 32;  // epilogue, TMA producer, MMA issuer

// Epilogues.
constexpr int kEpiLinear = 0;    // y = act(acc scales + bias) + residual, z before act
constexpr int kEpiPlain = 1;     // y = acc
constexpr int kEpiPartial32 = 2; // part[split] = acc in fp32 (split K)

struct LinearParams {
  CUtensorMap tm_a, tm_b;
  void* y;               // (M, N)
  void* z;               // nullable, (M, N)
  const void* residual;  // nullable, rows residual_stride apart
  int64_t residual_stride;
  const void* bias;              // nullable, (N)
  const uint8_t* a_scale;        // 8-bit operands: exponent bytes of A's and B's rows
  const uint8_t* b_scale;
  float* part;                   // kEpiPartial32: (k_splits, M, N)
  int32_t* header;               // nullable error word
  uint64_t handoff_limit_ns;     // of the wait for an accumulator to be read out
  int32_t M, N, K, k_splits;
  int32_t act;
  int32_t narrow;  // tiles of kTileN / 2 columns
};

template <int TN>
struct GemmSmem2 {
  alignas(1024) uint8_t a[kStages<TN>][kStageA];
  alignas(1024) uint8_t b[kStages<TN>][kStageB<TN>];
  alignas(8) uint64_t full[kStages<TN>], empty[kStages<TN>], acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort_flag;
  int issued[2];  // the leader's: stages that either CTA's producer loaded into
};
static_assert(sizeof(GemmSmem2<256>) + 1024 <= 232448 && sizeof(GemmSmem2<128>) + 1024 <= 232448, "over a CTA's shared memory");

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
// An arrival that orders nothing: what it reports, reads of TMEM, has completed (a
// releasing one waits until the warp's stores of results have reached L2, 2700 cycles).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Counts bytes that no copy brings as having come.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// 2-D load whose bytes are counted by a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// This thread's shared-memory writes become visible to MMAs and bulk copies.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 32 columns of 16 lanes of TMEM: value 4 g + 2 h + e of a lane of the warp is row
// lane / 4 + 8 h, column 8 g + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Word i of lane q of four becomes word q of lane i.
__device__ __forceinline__ void quad_transpose(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d, int q) {
  auto trade = [](uint32_t& low, uint32_t& high, bool upper, int with) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? low : high, with);
    low = upper ? got : low;
    high = upper ? high : got;
  };
  trade(a, b, q & 1, 1);
  trade(c, d, q & 1, 1);
  trade(a, c, q & 2, 2);
  trade(b, d, q & 2, 2);
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

// Waits until what the two producers loaded has landed, after an abort, which may have
// stopped them a stage apart: the leader arms a stage for the bytes of both CTAs, and either
// may be the one that issued its half alone. (No more than a stage of each barrier: a
// stage is loaded again only after both halves of its last load were multiplied.)
template <int RING>
__device__ __forceinline__ void settle_copies(uint64_t* full, const int* issued, uint32_t half) {
  const uint64_t t0 = globaltimer_ns();
  for (int st = 0; st < RING; ++st) {
    const uint32_t bar = smem_u32(&full[st]);
    const int leader = (issued[0] - st + RING - 1) / RING, other = (issued[1] - st + RING - 1) / RING;  // loads
    if (other > leader) mbar_expect_tx(bar, half);
    if (other < leader) mbar_complete_tx(bar, half);
    const int loads = max(leader, other);
    while (loads > 0 && !mbar_test(bar, (loads - 1) & 1) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
  }
}

// Loads ROWS rows (K-major, a box) or columns (MN-major) of an operand, one K block deep.
template <bool MN, int KB, int ROWS>
__device__ __forceinline__ void load_block(uint32_t dst, const CUtensorMap* map, uint32_t bar, int mn, int kb) {
  if (MN) {  // [64-column group][K row][128 bytes]
    tma_load_pair(dst, map, bar, mn, kb * KB);
    if (ROWS > 64) tma_load_pair(dst + 64 * 128, map, bar, mn + 64, kb * KB);
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
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + exp(-u)) of a pair; times x, u = x is SiLU, u = 2 sqrt(2 / pi) (x + 0.044715 x^3)
// the tanh form of GELU. The exponentials are of base 2 (argument m u, m = -log2(e)), and
// one reciprocal serves both values: 1 / a = b / (a b). (ex2 runs at 32 a cycle and SM,
// rcp at 16.) So that the product stays finite x counts as kLowest where it is
// below that: SiLU and GELU are -4e-17 and -6e-17 there, nearer to 0 below. A NaN
// stays with its own value.
constexpr float kGeluA = 1.5957691216057308f, kGeluB = 0.044715f;  // 2 sqrt(2 / pi)
constexpr float kLog2e = 1.4426950408889634f;
template <int ACT>
constexpr float kLowest = ACT == HSTU_ACT_GELU ? -7.3f : -41.5f;
__device__ __forceinline__ float max_nan(float x, float low) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(low));
  return r;
}
template <int ACT>
__device__ __forceinline__ uint64_t sigmoid_of(uint64_t x, uint64_t& e) {  // e: exp(-u)
  float a, b;
  pair_split(x, a, b);
  x = pair_of(fmaxf(a, kLowest<ACT>), fmaxf(b, kLowest<ACT>));  // NaN too
  uint64_t m;
  if (ACT == HSTU_ACT_SILU) {
    m = pair_mul(x, pair_of(-kLog2e, -kLog2e));
  } else {
    const uint64_t poly = pair_fma(pair_mul(x, x), pair_of(-kLog2e * kGeluA * kGeluB, -kLog2e * kGeluA * kGeluB),
                                   pair_of(-kLog2e * kGeluA, -kLog2e * kGeluA));
    m = pair_mul(x, poly);
  }
  pair_split(m, a, b);
  e = pair_of(exp2_fast(a), exp2_fast(b));
  pair_split(pair_add(e, pair_of(1.0f, 1.0f)), a, b);
  const float r = reciprocal_fast(a * b);
  return pair_mul(pair_of(r, r), pair_of(b, a));
}
template <int ACT>
__device__ __forceinline__ uint64_t activate2(uint64_t x) {
  if (ACT == HSTU_ACT_NONE) return x;
  float a, b;
  pair_split(x, a, b);
  constexpr float low = ACT == HSTU_ACT_RELU ? 0.0f : kLowest<ACT>;
  const uint64_t cut = pair_of(max_nan(a, low), max_nan(b, low));
  uint64_t e;
  return ACT == HSTU_ACT_RELU ? cut : pair_mul(cut, sigmoid_of<ACT>(x, e));
}

// Eight columns; nothing here reads them again.
__device__ __forceinline__ void store_cols(void* dst, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

template <typename T, bool F8, bool A_MN, bool B_MN, int EPI, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads2, 1)
    pair_gemm_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  GemmSmem2<TN>& s = *reinterpret_cast<GemmSmem2<TN>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int KB = F8 ? 128 : 64;  // K values of a block
  constexpr int kRing = kStages<TN>, kGroup = TN / 4;  // columns of an epilogue warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tm = (p.M + kTileM - 1) / kTileM, tn = (p.N + TN - 1) / TN;
  const int n_tiles = tm * tn * p.k_splits;
  const int nk = (p.K + KB - 1) / KB, per = (nk + p.k_splits - 1) / p.k_splits;
  // Tile t: K split t / (tm tn), then m tile, then n tile. Its K blocks are [kb0, kb1), one
  // at least.
  auto tile_of = [&](int t, int& m0, int& n0, int& split, int& kb0, int& kb1) {
    split = t / (tm * tn);
    const int rem = t - split * tm * tn;
    m0 = (rem / tn) * kTileM;
    n0 = (rem % tn) * TN;
    kb0 = min(split * per, nk);
    kb1 = min(kb0 + per, nk);
  };
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), 2 * kEpiWarps);  // of both CTAs
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
  }
  if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(smem_u32(&s.tmem_base), 2 * TN);
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
      int g = 0;
      bool ok = true;
      for (int t = pair; ok && t < n_tiles; t += pairs) {
        int m0, n0, split, kb0, kb1;
        tile_of(t, m0, n0, split, kb0, kb1);
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
          const int st = g % kRing, use = g / kRing;
          if (use > 0 && !mbar_wait(smem_u32(&s.empty[st]), (use - 1) & 1, abort_flag)) {
            store_cluster(peer_abort, 1);
            ok = false;
            break;
          }
          // The leader's barrier counts the bytes of both CTAs.
          if (rank == 0) mbar_expect_tx(smem_u32(&s.full[st]), 2 * (kStageA + kStageB<TN>));
          const uint32_t bar = in_cta(smem_u32(&s.full[st]), 0);
          load_block<A_MN, KB, 128>(smem_u32(s.a[st]), &p.tm_a, bar, m0 + 128 * rank, kb);
          load_block<B_MN, KB, TN / 2>(smem_u32(s.b[st]), &p.tm_b, bar, n0 + TN / 2 * rank, kb);
        }
      }
      store_cluster(in_cta(smem_u32(&s.issued[rank]), 0), g);
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0 && elect_one_sync()) {
      constexpr uint32_t idesc = idesc_f16kind(kTileM, TN, A_MN, B_MN, F8 ? 0u : Elem<T>::kUmma);
      int g = 0, i = 0;
      bool ok = true;
      for (int t = pair; ok && t < n_tiles; t += pairs, ++i) {
        int m0, n0, split, kb0, kb1;
        tile_of(t, m0, n0, split, kb0, kb1);
        const int buf = i & 1;
        // accumulator buf is free once both CTAs have read out tile i - 2 (a limit of 1 ns, set only by a
        // test, gives up at once, with copies and MMAs in flight)
        if (i >= 2) {
          ok = p.handoff_limit_ns > 1;
          if (!ok) *abort_flag = 1;
          ok = ok && mbar_wait(smem_u32(&s.acc_empty[buf]), ((i >> 1) - 1) & 1, abort_flag, p.handoff_limit_ns);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t tacc = tbase + buf * TN;
        for (int kb = kb0; kb < kb1; ++kb, ++g) {
          const int st = g % kRing;
          if (!mbar_wait(smem_u32(&s.full[st]), (g / kRing) & 1, abort_flag)) {
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
    // Warp w reads TMEM lanes 32 (w % 4) .. and columns TN / 4 (w / 4) .., in parts
    // of 32 columns: a lane gets two columns of each 8 of rows lane / 4 + 8 k, and the
    // lanes of four trade rounded results so that each has 8 columns of the rows; a
    // warp's loads and stores are runs of 64 bytes. Of 40960 rows, K = 512, N = 2048, with z
    // and SiLU: 75.6 us so, 78.9 us with the sums turned in shared memory, whose
    // bandwidth the operands take already (4096 of its cycles a tile, as long as their
    // MMAs); 87 us with 16-bit rows staged for TMA stores, 86 us with a row's 32-byte pieces
    // stored by its lane; 58 us without any stores, 45 us without an epilogue. What
    // it is short of now is the way out of the SM (requests to L2 69% of the cycles)
    // and, at 55%, issue slots.
    const int quarter = warp & 3, group = warp >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const int quad = lane & 3, sub_row = lane >> 2, sub_col = quad * 8;
    const int64_t skip = int64_t{8} * p.N;  // eight rows on
    bool ok = true;
    int i = 0;
    for (int t = pair; ok && t < n_tiles; t += pairs, ++i) {
      int m0, n0, split, kb0, kb1;
      tile_of(t, m0, n0, split, kb0, kb1);
      const int row0 = m0 + 128 * static_cast<int>(rank) + quarter * 32, col0 = n0 + group * kGroup;
      const int buf = i & 1, first_row = row0 + sub_row;
      const int rows = min(max((p.M - first_row + 7) >> 3, 0), 4);  // of the lane's four
      // What belongs to rows and columns is read while the accumulator is computed (the
      // first part's) or the part before is worked on.
      uint4 bias, residual[4];
      uint32_t col_scale[4];
      float row_scale[4];
      auto load_part = [&](int col) {
        if constexpr (EPI == kEpiLinear) {
          bias = make_uint4(0, 0, 0, 0);
          if (p.bias && col < p.N) bias = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + col);
          if (F8)
#pragma unroll
            for (int g = 0; g < 4; ++g) {  // of the lane's two columns of each eight
              const int at = col - sub_col + 8 * g;
              col_scale[g] = at < p.N ? *reinterpret_cast<const uint16_t*>(p.b_scale + at + 2 * quad) : 0u;
            }
          if (p.residual && col < p.N) {
            const T* from_row = static_cast<const T*>(p.residual) + first_row * p.residual_stride + col;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < rows) residual[k] = *reinterpret_cast<const uint4*>(from_row + 8 * k * p.residual_stride);
          }
        }
      };
      load_part(col0 + sub_col);
      if (EPI == kEpiLinear && p.residual && t + pairs < n_tiles) {
        // The next tile's rows, one a lane, come from HBM while this tile is computed.
        int m, n, sp, b0, b1;
        tile_of(t + pairs, m, n, sp, b0, b1);
        const int ahead = m + 128 * static_cast<int>(rank) + quarter * 32 + lane;
        if (ahead < p.M && n + group * kGroup < p.N)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T*>(p.residual) + ahead * p.residual_stride + n +
                                                        group * kGroup));
      }
      if (F8)
#pragma unroll
        for (int k = 0; k < 4; ++k) row_scale[k] = k < rows ? scale_value(p.a_scale[first_row + 8 * k]) : 0.0f;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.acc_full[buf]), (i >> 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      bool held = true;  // the accumulator
      auto release = [&] {
        tc_fence_before();
        if (lane == 0) arrive_cluster(in_cta(smem_u32(&s.acc_empty[buf]), 0));
        held = false;
      };
      // Two columns of each eight of the lane's four rows (a: as read), eight stored.
      auto write_part = [&](auto act, int col, const uint32_t (&a)[32]) {
        const int64_t at = static_cast<int64_t>(first_row) * p.N + col;
        if constexpr (EPI == kEpiLinear) quad_transpose(bias.x, bias.y, bias.z, bias.w, quad);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          [[maybe_unused]] const bool live = k < rows && col < p.N;
          const uint32_t* of = a + 16 * (k >> 1) + 2 * (k & 1);
          if constexpr (EPI == kEpiPartial32) {
            float* dst = p.part + static_cast<int64_t>(split) * p.M * p.N + at - sub_col + 2 * quad + k * skip;
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (k < rows && col - sub_col + 8 * g < p.N)
                asm volatile("st.global.L1::no_allocate.v2.b32 [%0], {%1, %2};" ::"l"(dst + 8 * g), "r"(of[4 * g]),
                             "r"(of[4 * g + 1])
                             : "memory");
          } else {
            uint64_t v[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) v[g] = pair_bits(of[4 * g], of[4 * g + 1]);
            auto store = [&](void* dst) {
              uint4 w = make_uint4(pack_pair<T>(v[0]), pack_pair<T>(v[1]), pack_pair<T>(v[2]), pack_pair<T>(v[3]));
              quad_transpose(w.x, w.y, w.z, w.w, quad);
              if (live) store_cols(static_cast<T*>(dst) + at + k * skip, w);
            };
            if constexpr (EPI == kEpiLinear) {
              const uint32_t bw[4] = {bias.x, bias.y, bias.z, bias.w};
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                if (F8) {  // w's scale first: that of a row with a mask's lowest value is 2^120, too much for a sum
                  v[g] = pair_mul(v[g], pair_of(scale_value(col_scale[g] & 0xffu), scale_value(col_scale[g] >> 8)));
                  v[g] = pair_mul(v[g], pair_of(row_scale[k], row_scale[k]));
                }
                v[g] = pair_add(v[g], unpack_pair<T>(bw[g]));
              }
              if (p.z) store(p.z);
#pragma unroll
              for (int g = 0; g < 4; ++g) v[g] = activate2<decltype(act)::value>(v[g]);
              if (p.residual) {
                uint4& w = residual[k];
                quad_transpose(w.x, w.y, w.z, w.w, quad);
                const uint32_t rw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int g = 0; g < 4; ++g) v[g] = pair_add(v[g], unpack_pair<T>(rw[g]));
              }
            }
            store(p.y);
          }
        }
      };
#pragma unroll
      for (int c = 0; c < kGroup / 32; ++c) {
        if (row0 >= p.M || col0 + 32 * c >= p.N) break;  // the same for the whole warp
        const int col = col0 + 32 * c + sub_col;
        uint32_t a[32];
        const uint32_t from = tbase + buf * TN + lane_addr + group * kGroup + c * 32;
        tmem_ld_rows16(from, a);
        tmem_ld_rows16(from + (16u << 16), a + 16);
        tmem_ld_wait(a);
        if (c == kGroup / 32 - 1) release();
        if constexpr (EPI == kEpiLinear) {
          switch (p.act) {
            case HSTU_ACT_SILU: write_part(std::integral_constant<int, HSTU_ACT_SILU>{}, col, a); break;
            case HSTU_ACT_GELU: write_part(std::integral_constant<int, HSTU_ACT_GELU>{}, col, a); break;
            case HSTU_ACT_RELU: write_part(std::integral_constant<int, HSTU_ACT_RELU>{}, col, a); break;
            default: write_part(std::integral_constant<int, HSTU_ACT_NONE>{}, col, a); break;
          }
        } else {
          write_part(std::integral_constant<int, HSTU_ACT_NONE>{}, col, a);
        }
        if (c < kGroup / 32 - 1) load_part(col + 32);
      }
      if (held) release();
      __syncwarp();
    }
    if (!ok && lane == 0) store_cluster(peer_abort, 1);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (rank == 1) mbar_wait_drain(smem_u32(&s.drain), 0);  // the last arrival that the leader's MMAs send here
    if (*abort_flag) store_cluster(peer_abort, 1);
  }
  __syncthreads();
  cluster_sync();  // nobody leaves while the other CTA's MMAs or arrivals may reach it; the flags are equal
  if (*abort_flag) {
    // Never leave with a copy in flight. (Without an abort the MMAs have waited for every one.)
    if (rank == 0 && threadIdx.x == 0) settle_copies<kRing>(s.full, s.issued, kStageA + kStageB<TN>);
    cluster_sync();
  }
  if (warp == kEpiWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 2 * TN);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.header) atomicOr(p.header + kHdrErr, kErrTimeout);
}

}  // namespace hstu

// Candidate rows against a paged K/V cache: the kernel (instantiated by
// paged_{bf16,f16}.cu, launched from paged.cu).
//
// For candidate c of sequence b: o = sum_j silu(alpha q.k_j) / N v_j over the
// visible cached positions j. Every cached row is read once and takes part in
// as many products as its sequence has candidates, few of them, so the bytes
// of the cache bound the kernel; the products run on warp-level matrix
// instructions (m16n8k16), whose operands a warp can take straight from the
// cache's rows.
//
// A CTA takes one (sequence, head) and one split of its length. Its four warps
// form slices of 1, 2 or 4 warps, as many as the sequence has groups of eight
// candidates; a slice reads every (4 / warps)-th step of 16 keys a warp into
// its ring of shared memory with asynchronous copies, and each of its warps
// multiplies all of the step's keys with its own eight candidates. Per 16 keys:
//   S = Q K^T   16 x 8 tiles, rows = 8 candidates (rows 8..15 see below)
//   P = silu(alpha S), zero where not visible, split into two 16-bit parts
//   O += P V    rows 0..7 hold the high part of P, rows 8..15 its low part
// With eight candidates in a 16-row operand the low part of P costs no extra
// instruction, and P V is as exact as with P in fp32 (rounding P to 16 bits
// instead would be as large an error as that of the output's own type).
//
// Operand layout. The order of the columns inside a contraction is free as
// long as both operands share it, so each lane reads whole 16-byte pieces of
// a row: lane (g, t) = (lane / 4, lane % 4) takes columns [8t, 8t + 8) of
// each 32 of key row g, which are its parts of two k = 16 steps, and the same
// columns of candidate row g. For P V lane (g, t) reads piece g of the key
// rows 2t, 2t+1, 2t+8, 2t+9 and pairs the rows' columns with byte
// permutations.
//
// Types. 16-bit caches multiply in their own type. 8-bit codes become fp16
// (exact); a bf16 candidate row is then scaled by a power of two and split
// into two fp16 parts in the same way as P (rows 8..15). A key's scale
// multiplies its column of S, a value row's scale its column of P, both exact
// powers of two. In fp16 the range of P needs care: a candidate's P is scaled
// by a power of two that follows its running maximum (when it grows, the sums
// so far are scaled down), which leaves 50 bits below the largest term.
#pragma once

#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "rope.cuh"

namespace hstu {

constexpr int kPagedWarps = 4;
constexpr int kPagedThreads = 32 * kPagedWarps;
constexpr int kPagedTile = 16;     // keys of a warp's step
constexpr int kPagedGroup = 8;     // candidates of a pass
constexpr int kPagedMaxSplit = 4096;  // keys of a split, at most

struct PagedParams {
  CacheView cache;
  const void* q;
  void* o;
  int64_t q_stride;
  const int32_t* lens;
  const int32_t* page_table;
  const int32_t* cand_offsets;  // null: candidate b belongs to sequence b
  const int32_t* func;          // null: everything cached is visible
  float* partial;
  int32_t* header;
  int32_t* counters;  // (batch, heads), zero at launch
  int32_t batch, max_pages, num_cand, nfunc, max_seqlen;
  int32_t split, nsplit;  // keys of a split; splits of max_seqlen
  float alpha, inv_n;
};

template <typename M>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// B bytes (16, 8 or 4) of a lane's piece, from shared memory.
template <int B>
__device__ __forceinline__ void load_piece(uint32_t addr, uint32_t* w) {
  if (B == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr));
  else if (B == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

// Asynchronous copy of 16 bytes; zeros where not live (src is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

__device__ __forceinline__ float silu_exact(float x) { return x * sigmoidf_fast(x); }

// Column `i` of a cached matrix as fp32 (8-bit codes without their scale).
template <typename T, bool E4M3>
__device__ __forceinline__ float cached_value(const void* base, int64_t i) {
  if (E4M3) return Elem<__half>::lo(e4m3x2_to_f16x2(static_cast<const uint8_t*>(base)[i]));
  return Elem<T>::lo(static_cast<const uint16_t*>(base)[i]);
}

// The sum of one candidate over the steps of one slice, in fp32, one visible
// key after the other: the way out for sums that are not finite. The slice
// takes entries [first, first + count), and so on every `stride` entries, of
// the split's list of 16-key tiles (the tiles themselves without a list).
template <typename T, int DQ, int DV, bool E4M3, int NI>
__device__ __noinline__ void paged_scalar_sum(const PagedParams& p, int cand, int h, int lane, int first, int count,
                                              int stride, int entries, const uint8_t* list, int k0, int k1, int len,
                                              const int* pages, float* out) {
  int lo[NI], hi[NI];
  if (p.func) {
    load_row_intervals<NI>(p.func, p.num_cand, cand, len, true, lo, hi, (1u << ((p.nfunc + 1) / 2)) - 1u);
  } else {
    for (int i = 0; i < NI; ++i) lo[i] = hi[i] = 0;
    hi[0] = len;
  }
  const uint16_t* q =
      static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(cand) * p.q_stride + static_cast<int64_t>(h) * DQ;
  const int page0 = k0 >> p.cache.page_shift;
  float sum[DV / 32];
  for (int i = 0; i < DV / 32; ++i) sum[i] = 0.0f;
  for (int e = first; e < entries; e = (e + 1 - first) % stride < count ? e + 1 : e + 1 + stride - count) {
    const int key0 = k0 + (p.func ? list[e] : e) * kPagedTile;
    const int64_t row0 = cache_row(p.cache, pages[(key0 >> p.cache.page_shift) - page0], h,
                                   key0 & ((1 << p.cache.page_shift) - 1));
    for (int key = key0; key < min(key0 + kPagedTile, k1); ++key) {
      bool vis = false;
      for (int i = 0; i < NI; ++i) vis |= lo[i] <= key && key < hi[i];
      if (!vis) continue;
      const int64_t row = row0 + key - key0;
      float dot = 0.0f;
      for (int i = lane; i < DQ; i += 32)
        dot = fmaf(Elem<T>::lo(q[i]), cached_value<T, E4M3>(p.cache.k, row * DQ + i), dot);
      for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (E4M3) dot *= scale_value(p.cache.k_scale[row]);
      float w = silu_exact(dot * p.alpha);
      if (E4M3) w *= scale_value(p.cache.v_scale[row]);
      for (int i = 0; i < DV / 32; ++i)
        sum[i] = fmaf(w, cached_value<T, E4M3>(p.cache.v, row * DV + lane + 32 * i), sum[i]);
    }
  }
  for (int i = 0; i < DV / 32; ++i) out[lane + 32 * i] = sum[i];
}

// Sizes that follow from the types and widths.
template <int DQ, int DV, bool E4M3>
struct PagedSizes {
  static constexpr int ES = E4M3 ? 1 : 2;               // bytes of a cached element
  static constexpr int KROW = DQ * ES, VROW = DV * ES;  // bytes of a cached row
  static constexpr int KC = KROW / 16, VC = VROW / 16;  // 16-byte pieces of a row
  // One warp's step: 16 rows of k, of v, and their scale bytes.
  static constexpr int kStep = kPagedTile * (KROW + VROW) + (E4M3 ? 32 : 0);
  // Steps in flight: enough bytes of the SM's CTAs together to cover HBM's
  // latency (48 KB an SM), within 227 KB of shared memory.
  static constexpr int kStages = kStep >= 8192 ? 3 : 4;
  static constexpr int kRing = kPagedWarps * kStages * kStep;
  static constexpr int kRed = kPagedWarps * kPagedGroup * DV * 4;  // the warps' sums, after the ring's use
  static constexpr int kSmem = kRing > kRed ? kRing : kRed;
  static constexpr int kResident = kSmem > 72 * 1024 ? 2 : 3;  // CTAs of an SM
};

// T: type of q, o and 16-bit pages. E4M3: 8-bit pages. NI: intervals a
// candidate may have.
template <typename T, int DQ, int DV, bool E4M3, int NI>
__global__ void __launch_bounds__(kPagedThreads, PagedSizes<DQ, DV, E4M3>::kResident) paged_kernel(const PagedParams p) {
  using Z = PagedSizes<DQ, DV, E4M3>;
  constexpr bool kHalf = E4M3 || std::is_same<T, __half>::value;  // products in fp16
  constexpr bool kSplitQ = E4M3 && !std::is_same<T, __half>::value;
  using M = typename std::conditional<kHalf, __half, __nv_bfloat16>::type;
  constexpr int KROW = Z::KROW, VROW = Z::VROW, KC = Z::KC, VC = Z::VC;
  // k pieces: a lane reads DQ / 4 columns of a key row
  constexpr int KB = (KROW / 4) < 16 ? KROW / 4 : 16;  // bytes of a piece
  constexpr int KP = KROW / 4 / KB;                    // pieces
  // v pieces: a lane reads DV / 8 columns of a key row
  constexpr int VB = (VROW / 8) < 16 ? VROW / 8 : 16;
  constexpr int VP = VROW / 8 / VB;
  constexpr int VE = VB / Z::ES;  // columns of a v piece
  constexpr int KSTEPS = DQ / 16, VTILES = DV / 8;
  constexpr float kLow = 2048.0f, kLowInv = 1.0f / 2048.0f;  // scale of the low parts in fp16
  constexpr float kMaxFinite = 3.402823466e38f;

  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int pages[kPagedMaxSplit / kPagedTile];
  __shared__ uint32_t tile_bits[kPagedMaxSplit / kPagedTile / 32];
  __shared__ uint8_t list[kPagedMaxSplit / kPagedTile];
  __shared__ int sh_flag, sh_entries;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t bid = blockIdx.x;
  const int split = static_cast<int>(bid % p.nsplit);
  const int bh = static_cast<int>(bid / p.nsplit);
  const int h = bh % p.cache.heads, b = bh / p.cache.heads;
  const int page_size = 1 << p.cache.page_shift;

  // Checks of this sequence (every CTA of it comes to the same answer).
  int cb = b, ce = b + 1;
  bool ok = true;
  if (p.cand_offsets) {
    cb = p.cand_offsets[b];
    ce = p.cand_offsets[b + 1];
    ok = cb >= 0 && cb <= ce && ce <= p.num_cand && p.cand_offsets[0] == 0 &&
         p.cand_offsets[p.batch] == p.num_cand;
  }
  const int len = p.lens[b];
  ok = ok && len >= 0 && len <= p.max_seqlen &&
       static_cast<int64_t>(len) <= (static_cast<int64_t>(p.max_pages) << p.cache.page_shift);
  if (!ok) {
    if (split == 0 && h == 0 && tid == 0) atomicOr(p.header + kHdrErr, kErrInput);
    return;
  }
  if (cb == ce) return;
  const int splits = max(1, (len + p.split - 1) / p.split);
  if (split >= splits) return;
  const int k0 = split * p.split, k1 = min(len, k0 + p.split);

  // Pages of this split.
  const int page0 = k0 >> p.cache.page_shift;
  const int npages = k1 > k0 ? ((k1 - 1) >> p.cache.page_shift) - page0 + 1 : 0;
  if (tid == 0) sh_flag = 0;
  __syncthreads();
  bool bad_page = false;
  for (int i = tid; i < npages; i += kPagedThreads) {
    const int pg = p.page_table[static_cast<int64_t>(b) * p.max_pages + page0 + i];
    pages[i] = pg;
    bad_page |= pg < 0 || pg >= p.cache.num_pages;
  }
  if (bad_page) sh_flag = 1;
  __syncthreads();
  const bool bad = sh_flag != 0;
  const int ntiles = bad ? 0 : (k1 - k0 + kPagedTile - 1) / kPagedTile;
  if (bad && tid == 0) atomicOr(p.header + kHdrErr, kErrInput);

  const char* kbase = static_cast<const char*>(p.cache.k);
  const char* vbase = static_cast<const char*>(p.cache.v);
  const uint32_t ring_addr = smem_u32(ring);
  float* red = reinterpret_cast<float*>(ring);

  for (int c0 = cb; c0 < ce;) {
    // Slices of `wg` warps; warp `gi` of its slice has candidates cg .. cg + 7.
    const int groups = (ce - c0 + kPagedGroup - 1) / kPagedGroup;
    const int wg = groups == 1 ? 1 : (groups == 2 ? 2 : 4);
    const int nslices = kPagedWarps / wg, slice = warp / wg, gi = warp % wg;
    const int cg = c0 + gi * kPagedGroup;
    const int ncand = max(0, min(kPagedGroup, ce - cg));
    const bool has = g < ncand;
    // Intervals of candidate g.
    int lo[NI], hi[NI];
    int entries = ntiles;
    if (p.func) {
      load_row_intervals<NI>(p.func, p.num_cand, cg + g, len, has, lo, hi, (1u << ((p.nfunc + 1) / 2)) - 1u);
      // The tiles that some candidate of this pass sees.
      if (tid < kPagedMaxSplit / kPagedTile / 32) tile_bits[tid] = 0;
      __syncthreads();
      if (slice == 0 && t == 0) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int a = max(lo[i], k0) - k0, e = min(hi[i], k1) - k0;
          if (e <= a) continue;
          const int first = a / kPagedTile, last = (e - 1) / kPagedTile;
          for (int w = first >> 5; w <= last >> 5; ++w) {
            uint32_t bits = 0xffffffffu;
            if (w == first >> 5) bits &= 0xffffffffu << (first & 31);
            if (w == last >> 5) bits &= 0xffffffffu >> (31 - (last & 31));
            atomicOr(&tile_bits[w], bits);
          }
        }
      }
      __syncthreads();
      if (warp == 0) {
        const uint32_t mine = (tile_bits[lane >> 2] >> (8 * (lane & 3))) & 0xffu;  // tiles 8 lane .. 8 lane + 7
        int at = __popc(mine);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, at, off);
          if (lane >= off) at += o;
        }
        if (lane == 31) sh_entries = bad ? 0 : at;
        at -= __popc(mine);
        for (int i = 0; i < 8; ++i)
          if ((mine >> i) & 1u) list[at++] = static_cast<uint8_t>(8 * lane + i);
      }
      __syncthreads();
      entries = sh_entries;
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) lo[i] = hi[i] = 0;
      if (has) hi[0] = len;
    }
    const int iters = (entries + kPagedWarps - 1) / kPagedWarps;

    // Copies this warp's tile of iteration `it` of its slice.
    const auto issue = [&](int it) {
      const int e = (it * nslices + slice) * wg + gi;
      if (it < iters && e < entries) {
        const int key0 = k0 + (p.func ? list[e] : e) * kPagedTile;
        const int page = pages[(key0 >> p.cache.page_shift) - page0];
        const int64_t row0 = cache_row(p.cache, page, h, key0 & (page_size - 1));
        const int nkeys = k1 - key0;
        const uint32_t dst = ring_addr + ((slice * Z::kStages + it % Z::kStages) * wg + gi) * Z::kStep;
        const char* ksrc = kbase + row0 * KROW;
        const char* vsrc = vbase + row0 * VROW;
#pragma unroll
        for (int i = 0; i < KROW / 32; ++i) {
          const int u = i * 32 + lane, r = u / KC, c = u % KC;
          const int sw = KC >= 8 ? (r & 1) << 2 : 0;
          copy16(dst + r * KROW + (c ^ sw) * 16, ksrc + u * 16, r < nkeys);
        }
#pragma unroll
        for (int i = 0; i < VROW / 32; ++i) {
          const int u = i * 32 + lane, r = u / VC, c = u % VC;
          const int sw = VC >= 8 ? r & 6 : (VC == 4 ? (r >> 1) & 3 : 0);
          copy16(dst + kPagedTile * KROW + r * VROW + (c ^ sw) * 16, vsrc + u * 16, r < nkeys);
        }
        if (E4M3 && lane < 2)
          copy16(dst + kPagedTile * (KROW + VROW) + 16 * lane, (lane ? p.cache.v_scale : p.cache.k_scale) + row0, true);
      }
      copies_commit();
    };
#pragma unroll
    for (int i = 0; i < Z::kStages - 1; ++i) issue(i);

    // Q fragments: rows 0..7 the candidates, rows 8..15 zero or low parts.
    uint32_t qa[KSTEPS][2], ql[kSplitQ ? KSTEPS : 1][2];
    float qscale = p.alpha;
    {
      const T* qrow = static_cast<const T*>(p.q) + static_cast<int64_t>(has ? cg + g : c0) * p.q_stride + h * DQ;
      constexpr int KE = KB / Z::ES;  // columns of a k piece: 16, 8
      float f[KSTEPS][4];
#pragma unroll
      for (int i = 0; i < KP; ++i) {
#pragma unroll
        for (int j = 0; j < KE / 4; ++j) {
          // columns of this lane in step (i * KE + 4 j) / 4: two for k 0..7, two for 8..15
          const int col = i * 4 * KE + t * KE + 4 * j;
          const uint2 u = has ? __ldg(reinterpret_cast<const uint2*>(qrow + col)) : make_uint2(0, 0);
          const int s = i * (KE / 4) + j;
          qa[s][0] = u.x;
          qa[s][1] = u.y;
          if (kSplitQ) {
            f[s][0] = Elem<T>::lo(u.x);
            f[s][1] = Elem<T>::hi(u.x);
            f[s][2] = Elem<T>::lo(u.y);
            f[s][3] = Elem<T>::hi(u.y);
          }
        }
      }
      if (kSplitQ) {
        uint32_t top = 0;  // largest magnitude of the row
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(f[s][e]) & 0x7fffffffu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(max(static_cast<int>(top >> 23), 27), 254);  // biased exponent
        const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);  // 2^(14 - (e - 127))
        qscale = p.alpha * __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const float x = f[s][2 * e2] * up, y = f[s][2 * e2 + 1] * up;
            const uint32_t w = pack_f16x2(x, y);
            qa[s][e2] = w;
            ql[s][e2] = pack_f16x2((x - Elem<__half>::lo(w)) * kLow, (y - Elem<__half>::hi(w)) * kLow);
          }
      }
    }

    float acc[VTILES][4];
#pragma unroll
    for (int j = 0; j < VTILES; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
    int erun = 30;  // biased exponent that this candidate's P is scaled to (fp16 products)

    for (int it = 0; it < iters; ++it) {
      copies_wait<Z::kStages - 2>();  // this warp's copies of iteration `it` have landed
      if (wg == 1) __syncwarp();
      else asm volatile("bar.sync %0, %1;" ::"r"(1 + slice), "r"(32 * wg) : "memory");
      issue(it + Z::kStages - 1);  // into the stage that the slice used last
      if (ncand == 0) continue;
      for (int j = 0; j < wg; ++j) {
        const int entry = (it * nslices + slice) * wg + j;
        if (entry >= entries) break;
        const int key0 = k0 + (p.func ? list[entry] : entry) * kPagedTile;
        const uint32_t kt = ring_addr + ((slice * Z::kStages + it % Z::kStages) * wg + j) * Z::kStep;
        const uint32_t vt = kt + kPagedTile * KROW;

        // S: key tile r holds keys 8r .. 8r + 7; this lane's columns are keys
        // 8r + 2t and 8r + 2t + 1 of candidate g.
        float s[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          s[r][0] = s[r][1] = s[r][2] = s[r][3] = 0.0f;
          const int row = g + 8 * r;
          const int sw = KC >= 8 ? (row & 1) << 2 : 0;
#pragma unroll
          for (int i = 0; i < KP; ++i) {
            uint32_t kw[KB / 4];
            const int byte = i * 4 * KB + t * KB;
            load_piece<KB>(kt + row * KROW + ((byte >> 4) ^ sw) * 16 + (byte & 15), kw);
            if (E4M3) {
#pragma unroll
              for (int w = 0; w < KB / 4; ++w) {
                const int st = i * (KB / 4) + w;
                mma16816<M>(s[r], qa[st][0], kSplitQ ? ql[kSplitQ ? st : 0][0] : 0u, qa[st][1],
                            kSplitQ ? ql[kSplitQ ? st : 0][1] : 0u, e4m3x2_to_f16x2(kw[w]),
                            e4m3x2_to_f16x2(kw[w] >> 16));
              }
            } else {
#pragma unroll
              for (int w = 0; w < KB / 8; ++w) {
                const int st = i * (KB / 8) + w;
                mma16816<M>(s[r], qa[st][0], 0u, qa[st][1], 0u, kw[2 * w], kw[2 * w + 1]);
              }
            }
          }
        }

        // P of candidate g at keys 2t, 2t+1, 2t+8, 2t+9.
        float pr[4];
        uint32_t scales[4];  // k and v scale bytes of keys 2t, 2t+1 and 2t+8, 2t+9
        if (E4M3) {
          const uint32_t sc = vt + kPagedTile * VROW + 2 * t;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            uint16_t u;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(sc + 8 * r));
            scales[r] = u;
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int key = key0 + 2 * t + (r & 1) + 8 * (r >> 1);
          float x = s[r >> 1][r & 1];
          if (kSplitQ) x = fmaf(s[r >> 1][2 + (r & 1)], kLowInv, x);
          x *= qscale;
          if (E4M3) x *= scale_value((scales[r >> 1] >> (8 * (r & 1))) & 0xffu);
          float v = silu_exact(x);
          if (E4M3) v *= scale_value((scales[2 + (r >> 1)] >> (8 * (r & 1))) & 0xffu);
          bool vis = false;
#pragma unroll
          for (int i = 0; i < NI; ++i) vis |= lo[i] <= key && key < hi[i];
          pr[r] = vis ? v : 0.0f;
        }
        uint32_t pa[2], pl[2];
        if (kHalf) {
          // Largest magnitude of the candidate in this tile: its four lanes.
          float top = fmaxf(fmaxf(fabsf(pr[0]), fabsf(pr[1])), fmaxf(fabsf(pr[2]), fabsf(pr[3])));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = static_cast<int>(__float_as_uint(top) >> 23);
          if (e > erun) {
            const float down = e - erun < 127 ? __uint_as_float(static_cast<uint32_t>(127 - (e - erun)) << 23) : 0.0f;
#pragma unroll
            for (int n = 0; n < VTILES; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[n][i] *= down;
            erun = e;
          }
          __syncwarp();
          const float up = __uint_as_float(static_cast<uint32_t>(268 - erun) << 23);  // 2^14 at the largest
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = pr[2 * r] * up, y = pr[2 * r + 1] * up;
            pa[r] = pack_f16x2(x, y);
            pl[r] = pack_f16x2((x - Elem<__half>::lo(pa[r])) * kLow, (y - Elem<__half>::hi(pa[r])) * kLow);
          }
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float x = pr[2 * r], y = pr[2 * r + 1];
            pa[r] = pack_bf16x2(x, y);
            pl[r] = pack_bf16x2(x - Elem<__nv_bfloat16>::lo(pa[r]), y - Elem<__nv_bfloat16>::hi(pa[r]));
          }
        }

        // O += P V: column tile (i, e) holds column e of the lanes' pieces i.
        // V rows 2t, 2t+1, 2t+8, 2t+9.
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          uint32_t vw[4][VB / 4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + 8 * (r >> 1);
            const int sw = VC >= 8 ? row & 6 : (VC == 4 ? (row >> 1) & 3 : 0);
            const int byte = i * 8 * VB + g * VB;
            load_piece<VB>(vt + row * VROW + ((byte >> 4) ^ sw) * 16 + (byte & 15), vw[r]);
          }
          if (E4M3) {
#pragma unroll
            for (int w = 0; w < VB / 4; ++w) {
              // bytes (row 0, row 1) of columns 4w, 4w+1 and 4w+2, 4w+3
              const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5140);
              const uint32_t x1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
              const uint32_t y0 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
              const uint32_t y1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
              float(*o)[4] = acc + i * VE + 4 * w;
              mma16816<M>(o[0], pa[0], pl[0], pa[1], pl[1], e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(y0));
              mma16816<M>(o[1], pa[0], pl[0], pa[1], pl[1], e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(y0 >> 16));
              mma16816<M>(o[2], pa[0], pl[0], pa[1], pl[1], e4m3x2_to_f16x2(x1), e4m3x2_to_f16x2(y1));
              mma16816<M>(o[3], pa[0], pl[0], pa[1], pl[1], e4m3x2_to_f16x2(x1 >> 16), e4m3x2_to_f16x2(y1 >> 16));
            }
          } else {
#pragma unroll
            for (int w = 0; w < VB / 4; ++w) {
              float(*o)[4] = acc + i * VE + 2 * w;
              mma16816<M>(o[0], pa[0], pl[0], pa[1], pl[1], __byte_perm(vw[0][w], vw[1][w], 0x5410),
                          __byte_perm(vw[2][w], vw[3][w], 0x5410));
              mma16816<M>(o[1], pa[0], pl[0], pa[1], pl[1], __byte_perm(vw[0][w], vw[1][w], 0x7632),
                          __byte_perm(vw[2][w], vw[3][w], 0x7632));
            }
          }
        }
      }
    }

    // This warp's sums: candidate g, columns (2t, 2t+1) of each column tile,
    // i.e. columns [2t VE, 2t VE + 2 VE) of piece group i.
    __syncthreads();  // the ring is free: the sums take its place
    float* mine = red + warp * kPagedGroup * DV;
    const float back = kHalf ? __uint_as_float(static_cast<uint32_t>(erun - 14) << 23) : 1.0f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < VP; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float(&a)[4] = acc[i * VE + e];
        const float x = (kHalf ? fmaf(a[2], kLowInv, a[0]) : a[0] + a[2]) * back;
        const float y = (kHalf ? fmaf(a[3], kLowInv, a[1]) : a[1] + a[3]) * back;
        finite = finite && fabsf(x) <= kMaxFinite && fabsf(y) <= kMaxFinite;
        mine[g * DV + i * 8 * VE + 2 * t * VE + e] = x;
        mine[g * DV + i * 8 * VE + (2 * t + 1) * VE + e] = y;
      }
    // A sum that is not finite may have met a value that its candidate does
    // not see (zero times infinity): those candidates are summed again, key by
    // key, over what they see alone.
    const uint32_t odd = __ballot_sync(0xffffffffu, has && !finite);
    if (odd != 0) {
      for (int r = 0; r < ncand; ++r)
        if (((odd >> (4 * r)) & 15u) != 0)
          paged_scalar_sum<T, DQ, DV, E4M3, NI>(p, cg + r, h, lane, slice * wg, wg, kPagedWarps, entries, list, k0, k1,
                                                len, pages, mine + r * DV);
    }
    __syncthreads();
    // The slices' sums in slice order.
    const int taken = min(ce - c0, wg * kPagedGroup);
    for (int i = tid; i < taken * DV; i += kPagedThreads) {
      const int r = i / DV, d = i % DV;
      const float* from = red + r * DV + d;  // group r / 8 is warp r / 8 of each slice
      float sum = from[0];
      for (int w = 1; w < nslices; ++w) sum += from[w * wg * kPagedGroup * DV];
      const int64_t at = static_cast<int64_t>(c0 + r) * p.cache.heads + h;
      if (splits > 1) {
        p.partial[(at * p.nsplit + split) * DV + d] = sum;
      } else if (!bad) {
        const uint32_t w = Elem<T>::pack2(sum * p.inv_n, 0.0f);
        static_cast<T*>(p.o)[at * DV + d] = *reinterpret_cast<const T*>(&w);
      }
    }
    __syncthreads();
    c0 += taken;
  }
  if (splits == 1) return;

  // The last CTA of this (sequence, head) to arrive joins the splits' sums in
  // a fixed order: a quarter of the splits for each warp, then the quarters.
  // A split with a bad page marks the counter, and nothing is written then.
  __threadfence();
  __syncthreads();
  if (tid == 0) sh_flag = atomicAdd(p.counters + bh, bad ? 1 + (1 << 20) : 1) + (bad ? 1 << 20 : 0);
  __syncthreads();
  const int seen = sh_flag;
  if ((seen & 0xfffff) != splits - 1 || seen >> 20 != 0) return;
  __threadfence();
  const int quarter = (splits + kPagedWarps - 1) / kPagedWarps;
  for (int c0 = cb; c0 < ce; c0 += kPagedGroup) {
    const int n = min(kPagedGroup, ce - c0);
    for (int item = warp; item < n * kPagedWarps; item += kPagedWarps) {
      const int r = item / kPagedWarps, qt = item % kPagedWarps;
      const float* from = p.partial + (static_cast<int64_t>(c0 + r) * p.cache.heads + h) * p.nsplit * DV;
      float sum[DV / 32];
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) sum[i] = 0.0f;
#pragma unroll 4
      for (int s = qt * quarter; s < min(splits, (qt + 1) * quarter); ++s)
#pragma unroll
        for (int i = 0; i < DV / 32; ++i) sum[i] += __ldcg(from + s * DV + 32 * i + lane);
#pragma unroll
      for (int i = 0; i < DV / 32; ++i) red[(qt * kPagedGroup + r) * DV + 32 * i + lane] = sum[i];
    }
    __syncthreads();
    for (int i = tid; i < n * DV; i += kPagedThreads) {
      float sum = red[i];
#pragma unroll
      for (int qt = 1; qt < kPagedWarps; ++qt) sum += red[qt * kPagedGroup * DV + i];
      const int64_t at = static_cast<int64_t>(c0 + i / DV) * p.cache.heads + h;
      const uint32_t w = Elem<T>::pack2(sum * p.inv_n, 0.0f);
      static_cast<T*>(p.o)[at * DV + i % DV] = *reinterpret_cast<const T*>(&w);
    }
    __syncthreads();
  }
}

// Launches the kernel for the widths of p.cache (one function for each type,
// in a translation unit of its own so that they compile in parallel).
template <typename T, bool E4M3, int DQ, int DV, int NI>
cudaError_t launch_paged_one(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  constexpr int kSmem = PagedSizes<DQ, DV, E4M3>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(paged_kernel<T, DQ, DV, E4M3, NI>, kSmem, done);
  if (e != cudaSuccess) return e;
  paged_kernel<T, DQ, DV, E4M3, NI><<<blocks, kPagedThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}
template <typename T, bool E4M3, int DQ, int DV>
cudaError_t launch_paged_widths(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  if (!p.func || p.nfunc == 1) return launch_paged_one<T, E4M3, DQ, DV, 1>(p, blocks, stream);
  return launch_paged_one<T, E4M3, DQ, DV, kMaxIntervals>(p, blocks, stream);
}
template <typename T, bool E4M3, int DQ>
cudaError_t launch_paged_dv(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  if (p.cache.dim_v == 128) return launch_paged_widths<T, E4M3, DQ, 128>(p, blocks, stream);
  if (p.cache.dim_v == 64) return launch_paged_widths<T, E4M3, DQ, 64>(p, blocks, stream);
  return launch_paged_widths<T, E4M3, DQ, 32>(p, blocks, stream);
}
template <typename T, bool E4M3>
cudaError_t launch_paged_typed(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  if (p.cache.dim == 128) return launch_paged_dv<T, E4M3, 128>(p, blocks, stream);
  if (p.cache.dim == 64) return launch_paged_dv<T, E4M3, 64>(p, blocks, stream);
  return launch_paged_dv<T, E4M3, 32>(p, blocks, stream);
}

cudaError_t launch_paged_bf16(const PagedParams& p, unsigned blocks, cudaStream_t stream);
cudaError_t launch_paged_f16(const PagedParams& p, unsigned blocks, cudaStream_t stream);
cudaError_t launch_paged_bf16_e4m3(const PagedParams& p, unsigned blocks, cudaStream_t stream);
cudaError_t launch_paged_f16_e4m3(const PagedParams& p, unsigned blocks, cudaStream_t stream);

}  // namespace hstu

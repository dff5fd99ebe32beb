// Candidate rows against a paged K/V cache: the kernel (instantiated by
// paged_{bf16,f16}{,_e4m3}.cu, launched from paged.cu).
//
// For candidate c of sequence b: o = sum_j silu(alpha q.k_j) / N v_j over the
// visible cached positions j. A cached row is read once for each 64 candidates of
// its sequence (a pass) and takes part in as many products as the pass has
// candidates, few of them, so the bytes of the cache bound the kernel; the
// products run on warp-level matrix instructions (m16n8k16), whose operands a
// warp can take straight from the cache's rows. (Where sequences have more than
// 16 candidates on average the products are worth tcgen05's operand tiles in
// shared memory, for the types, widths and lengths that paged.cu's
// paged_layout names: paged_many.cuh.)
//
// Measured, H = 4, D_qk = D_v = 128, histories of 1332 to 3994 rows: one
// candidate for each of 256 users over 16-bit pages 207 us, 6.8 TB/s, the rate of
// a plain copy; over 8-bit pages 118 us, 6.0 TB/s, with the issue slots half
// used by the codes' conversion and the latency of the first and last CTAs. 16
// candidates for each of 64 users of 512 to 2048 rows: 47 us against 25 us for the
// bytes, bound by the latency of the chain from scores to weights in the twelve
// warps that registers leave an SM and by the CTAs' first loads.
//
// A CTA takes one (sequence, head) and one split of its length. Its four warps
// form slices of 1, 2 or 4 warps, as many as the sequence's candidates need; a
// warp reads tiles of 16 keys into its ring of shared memory with asynchronous
// copies, and each warp of a slice multiplies all of the slice's tiles with
// its own candidates. Per tile, keys and value columns as the 16 rows of the
// products and candidates as their 8 columns:
//   S^T = K Q^T    P = silu(alpha S), zero where not visible
//   O^T += V^T P^T P in two 16-bit parts, which leave a relative error of 2^-17 in
//                  bf16 and 2^-23 in fp16 (fp32: 2^-24); one part alone would be
//                  off by as much as the output's own rounding to that type
//                  (2^-8, 2^-11)
// Up to four candidates ("pair") have two columns each, one for each part of
// P, so that one instruction adds both. More ("full") take a column each, in
// one or two groups of eight, and an instruction for each part: a piece of K
// and V that is brought into operand form then serves up to 16 candidates.
//
// Operand layout. The order of the columns inside a contraction is free as
// long as both operands share it, so each lane reads whole 16-byte pieces of
// a row: lane (g, t) = (lane / 4, lane % 4) takes columns [8t, 8t + 8) of
// each 32 of key rows g and g + 8, which are its parts of two k = 16 steps, and
// the same columns of candidate row g. 16-bit value rows are transposed by
// ldmatrix. Of 8-bit ones the lane reads piece g of the key rows 2t, 2t+1, 2t+8,
// 2t+9 and pairs the rows' columns with byte permutations. P^T comes out of the
// first product with keys along g and is turned by movmatrix, 8 x 8 values an
// instruction. In shared memory the 16-byte pieces of a row are permuted by
// bits of the row's index so that the lanes of a load phase meet different
// banks.
//
// Types. 16-bit caches multiply in their own type. 8-bit codes become fp16
// (exact); a bf16 candidate row is then scaled by a power of two and split
// into two fp16 parts in the same way as P. A key's scale
// multiplies its column of S, a value row's scale its column of P, both exact
// powers of two. In fp16 the range of P needs care: a candidate's P is scaled
// by a power of two that follows its running maximum (when it grows, the sums
// so far are scaled down), which leaves 39 bits below the largest term.
#pragma once

#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "rope.cuh"

namespace hstu {

constexpr int kPagedWarps = 4;       // of a CTA
constexpr int kPagedWarpsWide = 8;  // and where there is no more than one CTA an SM
constexpr int kPagedTile = 16;     // keys of a warp's step
constexpr int kPagedPass = 64;     // candidates of a pass, at most
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
  int32_t* header;    // null: bad sequences are not reported
  int32_t* states;    // (batch, heads, nsplit): 1 where a split's sums are good
  int32_t batch, max_pages, num_cand, nfunc, max_seqlen;
  int32_t split, nsplit;  // keys of a split (of sequences with few candidates); splits of max_seqlen, at most
  bool tensor;            // many candidates: paged_many_kernel
  bool zero;              // rows that would be left as they were become zeros
  bool shorter;           // splits get shorter with a sequence's candidates (paged_split_keys)
  float alpha, inv_n;
  bool give_up;  // set by a test: paged_many_kernel takes its way out of a wait that ran out
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
__device__ __forceinline__ void load_piece(const uint8_t* p, uint32_t* w) {
  if (B == 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  } else if (B == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Four 8 x 8 blocks of 16-bit values, each transposed: lane l gives the address
// of row l % 8 of block l / 8.
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t (&w)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr));
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

// x sigmoid(x) with the hardware's exponential and reciprocal (relative error
// about |x| 2^-24 + 2^-22). Far below zero the exponential is infinite and the
// result -0.
__device__ __forceinline__ float silu_exact(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return x * r;
}

// Column `i` of a cached matrix as fp32 (8-bit codes without their scale).
template <typename T, bool E4M3>
__device__ __forceinline__ float cached_value(const void* base, int64_t i) {
  if (E4M3) return Elem<__half>::lo(e4m3x2_to_f16x2(static_cast<const uint8_t*>(base)[i]));
  return Elem<T>::lo(static_cast<const uint16_t*>(base)[i]);
}

// Sizes that follow from the types and widths. MANY: the kernel for any number
// of candidates; otherwise the one for a single candidate a sequence.
template <int DQ, int DV, bool E4M3, bool MANY, int W = kPagedWarps>
struct PagedSizes {
  static constexpr int kWarps = W, kThreads = 32 * W;
  static constexpr int ES = E4M3 ? 1 : 2;               // bytes of a cached element
  static constexpr int KROW = DQ * ES, VROW = DV * ES;  // bytes of a cached row
  static constexpr int KC = KROW / 16, VC = VROW / 16;  // 16-byte pieces of a row
  // k pieces: a lane reads KP of KB bytes, DQ / 4 columns of a key row;
  // v pieces: VP of VB bytes (VE columns), DV / 8 columns of a key row
  static constexpr int KB = KROW / 4 < 16 ? KROW / 4 : 16, KP = KROW / 4 / KB;
  static constexpr int VB = VROW / 8 < 16 ? VROW / 8 : 16, VP = VROW / 8 / VB, VE = VB / ES;
  // One warp's tile: 16 rows of k, of v, and their scale bytes.
  static constexpr int kStep = kPagedTile * (KROW + VROW) + (E4M3 ? 32 : 0);
  // Tiles of a warp's ring: enough in flight on an SM to cover HBM's latency
  // (48 KB); two stages where the warps of a slice share tiles, whose products
  // take longer than the copies.
  static constexpr int kStages = kStep <= 2080 ? 4 : (MANY && kStep >= 4096) || kStep == 6144 ? 2 : 3;
  static constexpr int kRing = W * kStages * kStep;
  // The warps' sums, after the ring's use. A lane (g, t) writes VE columns of
  // each piece of row t: blocks of VE + 1 and rows of 8 (mod 32) put the
  // lanes' stores into different banks.
  // (16-bit pages: columns g and g + 8 of each 16, no padding needed.)
  static constexpr int kBlock = VE + 1;
  static constexpr int kRedRow = E4M3 ? (VP * 8 * kBlock + 31) / 32 * 32 + 8 : DV + 8;
  static constexpr int kRedRows = MANY ? 16 : 4;  // of a warp
  static constexpr int kRed = W * kRedRows * kRedRow * 4;
  static constexpr int kSmem = kRing > kRed ? kRing : kRed;
  // CTAs of an SM: as many as shared memory has room for, up to 4 (3 to 5 for
  // many candidates, whose sums and fragments are most of the registers).
  static constexpr int kFit = 227 * 1024 / (kSmem + 6144);
  static constexpr int kRegisters = 80 + DV / 2 + DQ / 4 * (E4M3 ? 2 : 1);
  static constexpr int kWant =
      !MANY ? (W == kPagedWarps ? 4 : 2) : (kRegisters <= 102 ? 5 : (kRegisters <= 128 ? 4 : 3));
  static constexpr int kResident = kFit < 1 ? 1 : (kFit > kWant ? kWant : kFit);
  static __device__ __forceinline__ int red_column(int d) { return E4M3 ? d / VE * kBlock + d % VE : d; }
  // Permutation of the 16-byte pieces of v row r.
  static __device__ __forceinline__ int v_swizzle(int r) {
    if (!E4M3) return VC >= 8 ? r & 7 : (r >> 1) & 3;
    return VC >= 8 ? r & 6 : (VC == 4 ? (r >> 1) & 3 : 0);
  }
};

extern __shared__ __align__(128) uint8_t paged_ring[];

// What a CTA's passes share.
struct PagedSplit {
  int h, k0, k1, len, page0, tiles;
  int c0, ce;         // candidates still to do
  const int* pages;   // shared memory: pages of the split,
  uint32_t* bits;     // tiles that some candidate sees, tiles that some does not see whole,
  uint16_t* list;     // the seen tiles (bit 15: not seen whole by all)
  int* iv;            // and the candidates' intervals
  int* entries;
  uint32_t ring;      // shared-memory address of the ring
  float* red;
};
constexpr int kPagedWords = kPagedMaxSplit / kPagedTile / 32;
constexpr int kPagedIv = 2 * kMaxIntervals + 1;  // ints of a candidate's intervals (odd: different banks)

// The bits of a word of 32 tiles whose tiles lie in [x, y).
__device__ __forceinline__ uint32_t tile_span(int x, int y) {
  const int u = max(x, 0), v = min(y, 32);
  return u >= v ? 0u : (0xffffffffu << u) & (0xffffffffu >> (32 - v));
}

// Tiles of word w that the intervals touch (seen) and that one of them covers.
__device__ __forceinline__ void tile_words(const PagedSplit& sp, int w, const int (&lo)[kMaxIntervals],
                                           const int (&hi)[kMaxIntervals], int n, uint32_t& seen, uint32_t& whole) {
  const int base = sp.k0 + w * 32 * kPagedTile;
  seen = whole = 0;
#pragma unroll
  for (int i = 0; i < kMaxIntervals; ++i) {
    if (i >= n) break;
    const int a = max(lo[i], sp.k0) - base, e = min(hi[i], sp.k1) - base;  // in keys of the word's first tile
    if (e <= a) continue;
    seen |= tile_span(a >> 4, (e + kPagedTile - 1) >> 4);
    whole |= tile_span((a + kPagedTile - 1) >> 4, e >> 4);
  }
}

// The n intervals of a candidate from its raw values, cut to [0, len); empty
// ones are [0, 0).
__device__ __forceinline__ void paged_intervals(const int (&raw)[2 * kMaxIntervals - 1], int len, int n,
                                                int (&lo)[kMaxIntervals], int (&hi)[kMaxIntervals]) {
#pragma unroll
  for (int i = 0; i < kMaxIntervals; ++i) {
    lo[i] = i == 0 ? 0 : min(max(raw[i > 0 ? 2 * i - 1 : 0], 0), len);
    hi[i] = min(max(raw[2 * i], 0), len);
    if (i >= n || hi[i] <= lo[i]) lo[i] = hi[i] = 0;
  }
}

// Lists the tiles that the pass's candidates see. A single candidate's raw
// intervals are in every thread's registers.
template <bool MANY>
__device__ __forceinline__ int paged_list(const PagedParams& p, const PagedSplit& sp, int ncand,
                                          const int (&raw)[2 * kMaxIntervals - 1]) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int words = (sp.tiles + 31) / 32, n = (p.nfunc + 1) / 2;
  int lo[kMaxIntervals], hi[kMaxIntervals];
  if (MANY) {
    if (tid < 2 * kPagedWords) sp.bits[tid] = 0;
    __syncthreads();
    if (tid < ncand) {
      int mine[2 * kMaxIntervals - 1];
#pragma unroll
      for (int i = 0; i < 2 * kMaxIntervals - 1; ++i)
        mine[i] = i < p.nfunc ? p.func[static_cast<int64_t>(i) * p.num_cand + sp.c0 + tid] : 0;
      paged_intervals(mine, sp.len, n, lo, hi);
      for (int w = 0; w < words; ++w) {
        uint32_t seen, whole;
        tile_words(sp, w, lo, hi, n, seen, whole);
        if (seen) atomicOr(sp.bits + w, seen);
        if (~whole) atomicOr(sp.bits + kPagedWords + w, ~whole);
      }
    }
  } else {
    paged_intervals(raw, sp.len, n, lo, hi);
    if (tid < kPagedWords) {
      uint32_t seen = 0, whole = 0;
      if (tid < words) tile_words(sp, tid, lo, hi, n, seen, whole);
      sp.bits[tid] = seen;
      sp.bits[kPagedWords + tid] = ~whole;
    }
  }
  if (tid < ncand) {
#pragma unroll
    for (int i = 0; i < kMaxIntervals; ++i) {
      if (i >= n) break;
      sp.iv[tid * kPagedIv + 2 * i] = lo[i];
      sp.iv[tid * kPagedIv + 2 * i + 1] = hi[i];
    }
  }
  __syncthreads();
  if (tid < 32) {
    const int shift = 8 * (lane & 3);
    const uint32_t mine = (sp.bits[lane >> 2] >> shift) & 0xffu;  // tiles 8 lane .. 8 lane + 7
    const uint32_t part = (sp.bits[kPagedWords + (lane >> 2)] >> shift) & 0xffu;
    int at = __popc(mine);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, at, off);
      if (lane >= off) at += o;
    }
    if (lane == 31) *sp.entries = sp.tiles > 0 ? at : 0;
    at -= __popc(mine);
    for (int i = 0; i < 8; ++i)
      if ((mine >> i) & 1u) sp.list[at++] = static_cast<uint16_t>((8 * lane + i) | (((part >> i) & 1u) << 15));
  }
  __syncthreads();
  return *sp.entries;
}

// Whether candidate r of the pass sees `key`.
__device__ __forceinline__ bool paged_sees(const PagedParams& p, const PagedSplit& sp, int r, int key) {
  if (!p.func) return key < sp.k1;
  bool vis = false;
  const int n = (p.nfunc + 1) / 2;
  for (int i = 0; i < n; ++i) vis |= sp.iv[r * kPagedIv + 2 * i] <= key && key < sp.iv[r * kPagedIv + 2 * i + 1];
  return vis;
}

// Warps of a slice for `total` candidates of a pass.
__host__ __device__ __forceinline__ int paged_slice(int total) { return total <= 16 ? 1 : (total <= 32 ? 2 : 4); }

// Keys of a split of a sequence with `total` candidates: where the warps of a
// slice share their tiles, each takes all of them, so the split is shorter by
// as much and CTAs take about the same time.
__device__ __forceinline__ int paged_split_keys(const PagedParams& p, int total) {
  return p.shorter ? p.split / paged_slice(total) : p.split;
}

__device__ __forceinline__ int paged_key(const PagedParams& p, const PagedSplit& sp, int entry) {
  return sp.k0 + (p.func ? sp.list[entry] & 0x7fff : entry) * kPagedTile;
}

// What a CTA keeps in shared memory besides its tiles.
template <bool MANY>
struct PagedTables {
  int pages[kPagedMaxSplit / kPagedTile];
  uint32_t bits[2 * kPagedWords];
  uint16_t list[kPagedMaxSplit / kPagedTile];
  int iv[(MANY ? kPagedPass : 1) * kPagedIv];
  int entries;
};

// Zeros in head h of candidate rows [first, last), by all threads of the CTA.
inline __device__ __noinline__ void paged_zero_rows(void* o, int heads, int dim_v, int h, int64_t first, int64_t last) {
  const int pieces = dim_v / 8;  // of 16 bytes
  for (int64_t i = threadIdx.x; i < (last - first) * pieces; i += blockDim.x)
    static_cast<uint4*>(o)[((first + i / pieces) * heads + h) * pieces + i % pieces] = make_uint4(0, 0, 0, 0);
}

// Opens one split, of `keys` keys, of sequence b for candidates [cb, ce): reads its
// pages and checks the sequence. False where there is nothing to do; `bad`
// where a page of the split is no page of the cache (it has no tiles then).
template <bool MANY, int THREADS>
__device__ __forceinline__ bool paged_open(const PagedParams& p, PagedTables<MANY>& tables, int b, int h, int split,
                                           int cb, int ce, int keys, PagedSplit& sp, int& splits, bool& bad) {
  const int tid = threadIdx.x;
  // Loads that depend on nothing, all under way at once.
  const int len = p.lens[b];
  const int offsets0 = MANY ? p.cand_offsets[0] : 0, offsets1 = MANY ? p.cand_offsets[p.batch] : p.num_cand;
  const int k0 = static_cast<int>(min(static_cast<int64_t>(split) * keys, static_cast<int64_t>(p.max_seqlen)));

  // Pages of this split, read before the length is known (entries past the
  // length are not looked at).
  const int page0 = k0 >> p.cache.page_shift;
  const int most_pages = min(((k0 + keys - 1) >> p.cache.page_shift) - page0 + 1, p.max_pages - page0);
  constexpr int kPageLoads = (kPagedMaxSplit / kPagedTile + THREADS - 1) / THREADS;
  int page[kPageLoads];
#pragma unroll
  for (int i = 0; i < kPageLoads; ++i) {
    const int at = i * THREADS + tid;
    page[i] = at < most_pages ? p.page_table[static_cast<int64_t>(b) * p.max_pages + page0 + at] : -1;
  }
  // Checks of this sequence (every CTA of it comes to the same answer).
  bool ok = true;
  if (MANY) ok = (cb >= 0) & (cb <= ce) & (ce <= p.num_cand) & (offsets0 == 0) & (offsets1 == p.num_cand);
  ok = ok && len >= 0 && len <= p.max_seqlen &&
       static_cast<int64_t>(len) <= (static_cast<int64_t>(p.max_pages) << p.cache.page_shift);
  if (!ok) {
    if (p.header && split == 0 && h == 0 && tid == 0) atomicOr(p.header + kHdrErr, kErrInput);
    if (p.zero && split == 0) {
      // Offsets with a wrong end make every sequence bad, and each takes a share
      // of all rows. With right ends every row lies between the offsets of some
      // sequence, a bad one among them reaching past the ends at the most.
      const bool ends = offsets0 == 0 && offsets1 == p.num_cand;
      const int64_t rows = p.num_cand;
      paged_zero_rows(p.o, p.cache.heads, p.cache.dim_v, h, ends ? max(cb, 0) : rows * b / p.batch,
                      ends ? min(ce, p.num_cand) : rows * (b + 1) / p.batch);
    }
    return false;
  }
  if (cb == ce) return false;
  splits = max(1, (len + keys - 1) / keys);
  if (split >= splits) return false;
  const int k1 = min(len, k0 + keys);
  const int npages = k1 > k0 ? ((k1 - 1) >> p.cache.page_shift) - page0 + 1 : 0;
  bool bad_page = false;
#pragma unroll
  for (int i = 0; i < kPageLoads; ++i) {
    const int at = i * THREADS + tid;
    if (at < npages) {
      tables.pages[at] = page[i];
      bad_page |= page[i] < 0 || page[i] >= p.cache.num_pages;
    }
  }
  bad = __syncthreads_or(bad_page) != 0;
  if (bad && p.header && tid == 0) atomicOr(p.header + kHdrErr, kErrInput);
  sp.h = h;
  sp.k0 = k0;
  sp.k1 = k1;
  sp.len = len;
  sp.page0 = page0;
  sp.tiles = bad ? 0 : (k1 - k0 + kPagedTile - 1) / kPagedTile;
  sp.ce = ce;
  sp.pages = tables.pages;
  sp.bits = tables.bits;
  sp.list = tables.list;
  sp.iv = tables.iv;
  sp.entries = &tables.entries;
  return true;
}

// The sum of candidate r of the pass over the tiles of one slice, in fp32, one
// visible key after the other: the way out for sums that are not finite. The
// slice takes entries [first, first + count), and so on every `Z::kWarps` entries.
template <typename T, int DQ, int DV, bool E4M3, typename Z>
__device__ __noinline__ void paged_scalar_sum(const PagedParams& p, const PagedSplit& sp, int r, int first, int count,
                                              int entries, float* out) {
  const int lane = threadIdx.x & 31;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + static_cast<int64_t>(sp.c0 + r) * p.q_stride +
                      static_cast<int64_t>(sp.h) * DQ;
  float sum[DV / 32];
  for (int i = 0; i < DV / 32; ++i) sum[i] = 0.0f;
  for (int e = first; e < entries;
       e = (e + 1 - first) % Z::kWarps < count ? e + 1 : e + 1 + Z::kWarps - count) {
    const int key0 = paged_key(p, sp, e);
    const int64_t row0 = cache_row(p.cache, sp.pages[(key0 >> p.cache.page_shift) - sp.page0], sp.h,
                                   key0 & ((1 << p.cache.page_shift) - 1));
    for (int key = key0; key < min(key0 + kPagedTile, sp.k1); ++key) {
      if (!paged_sees(p, sp, r, key)) continue;
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
  for (int i = 0; i < DV / 32; ++i) out[Z::red_column(lane + 32 * i)] = sum[i];
}

// 8 x 8 16-bit values, row g columns 2t, 2t+1 in lane (g, t), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

// One pass over the split's keys: the sums of candidates c0 .. of this
// sequence, as many as fit, in the CTA's shared memory. PAIR: two columns for
// each of up to 4 candidates; otherwise two groups of eight columns a warp (the
// second idle where a warp has 8 candidates or fewer). Returns the warps of a
// slice.
template <typename T, int DQ, int DV, bool E4M3, bool MANY, int W, bool PAIR>
__device__ __forceinline__ int paged_pass(const PagedParams& p, const PagedSplit& sp,
                                          const int (&raw)[2 * kMaxIntervals - 1]) {
  using Z = PagedSizes<DQ, DV, E4M3, MANY, W>;
  constexpr bool kPair = PAIR;
  constexpr bool kHalf = E4M3 || std::is_same<T, __half>::value;  // products in fp16
  constexpr bool kSplitQ = E4M3 && !std::is_same<T, __half>::value;
  using M = typename std::conditional<kHalf, __half, __nv_bfloat16>::type;
  constexpr int KROW = Z::KROW, VROW = Z::VROW, KC = Z::KC, VC = Z::VC;
  constexpr int KB = Z::KB, KP = Z::KP, VB = Z::VB, VP = Z::VP, VE = Z::VE;
  constexpr int KSTEPS = DQ / 16, VTILES = DV / 16, S = Z::kStages;
  constexpr int NG = kPair ? 1 : 2;      // column groups
  constexpr int NC = kPair ? 1 : 4;      // candidates of a lane
  constexpr int ROWS = kPair ? 4 : 16;   // candidates of a warp
  constexpr float kMaxFinite = 3.402823466e38f;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int total = sp.ce - sp.c0;
  const int wg = kPair ? 1 : paged_slice(total);
  const int nslices = W / wg, slice = warp / wg, gi = warp % wg;
  const int cg = gi * ROWS;                                        // this warp's first candidate in the pass
  const int ncand = max(0, min(ROWS, total - cg));
  const int groups = kPair ? 1 : (ncand > 8 ? 2 : 1);              // column groups in use
  const int entries = p.func ? paged_list<MANY>(p, sp, min(total, wg * ROWS), raw) : sp.tiles;
  // Copy n of this warp is list entry (n nslices + slice) wg + gi.
  const int iters = (entries + W - 1) / W;

  const uint32_t ring = sp.ring + slice * S * wg * Z::kStep;  // the slice's stages
  const auto issue = [&](int n, int stage) {
    const int e = (n * nslices + slice) * wg + gi;
    if (n < iters && e < entries) {
      const int key0 = paged_key(p, sp, e);
      const int page = sp.pages[(key0 >> p.cache.page_shift) - sp.page0];
      const int64_t row0 = cache_row(p.cache, page, sp.h, key0 & ((1 << p.cache.page_shift) - 1));
      const int nkeys = sp.k1 - key0;  // zeros behind the last key
      const uint32_t dst = ring + (stage * wg + gi) * Z::kStep;
      const char* ksrc = static_cast<const char*>(p.cache.k) + row0 * KROW + lane * 16;
      const char* vsrc = static_cast<const char*>(p.cache.v) + row0 * VROW + lane * 16;
#pragma unroll
      for (int i = 0; i < KROW / 32; ++i) {
        const int u = i * 32 + lane, r = u / KC, c = u % KC;
        const int sw = KC >= 8 ? (r & 1) << 2 : 0;
        copy16(dst + r * KROW + (c ^ sw) * 16, ksrc + i * 512, r < nkeys);
      }
#pragma unroll
      for (int i = 0; i < VROW / 32; ++i) {
        const int u = i * 32 + lane, r = u / VC, c = u % VC;
        copy16(dst + kPagedTile * KROW + r * VROW + (c ^ Z::v_swizzle(r)) * 16, vsrc + i * 512, r < nkeys);
      }
      if (E4M3 && lane < 2)
        copy16(dst + kPagedTile * (KROW + VROW) + 16 * lane, (lane ? p.cache.v_scale : p.cache.k_scale) + row0, true);
    }
    copies_commit();
  };
  // The first S - 1 copies run while Q is loaded.
#pragma unroll 1
  for (int n = 0; n < S - 1; ++n) issue(n, n);

  // Q fragments, column g of each group. 8-bit caches with bf16 rows: two fp16
  // parts of the row scaled to a largest magnitude of 2^14 to 2^15, which is
  // put right in qscale (of this lane's candidates in the scores).
  uint32_t qa[NG][KSTEPS][2], ql[kSplitQ && !kPair ? NG : 1][kSplitQ && !kPair ? KSTEPS : 1][2];
  float qscale[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) qscale[c] = p.alpha;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const int r = kPair ? g >> 1 : 8 * n + g;
    const bool has = r < ncand && (!kPair || kSplitQ || (g & 1) == 0);
    const T* qrow = static_cast<const T*>(p.q) + static_cast<int64_t>(sp.c0 + (has ? cg + r : 0)) * p.q_stride +
                    static_cast<int64_t>(sp.h) * DQ;
    constexpr int KE = KB / Z::ES;  // columns of a k piece
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < KP; ++i) {
#pragma unroll
      for (int j = 0; j < KE / 4; ++j) {
        // columns of this lane in step st: two for k 0..7, two for 8..15
        const int st = i * (KE / 4) + j;
        const uint2 u =
            has ? *reinterpret_cast<const uint2*>(qrow + i * 4 * KE + t * KE + 4 * j) : make_uint2(0, 0);
        qa[n][st][0] = u.x;
        qa[n][st][1] = u.y;
        if (kSplitQ)
          top = max(max(top, max((u.x << 16) & 0x7fff0000u, u.x & 0x7fff0000u)),
                    max((u.y << 16) & 0x7fff0000u, u.y & 0x7fff0000u));
      }
    }
    if (kSplitQ) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max(static_cast<int>(top >> 23), 27), 254);            // biased exponent
      const float up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);  // 2^(14 - (e - 127))
      const float back = p.alpha * __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
#pragma unroll
      for (int st = 0; st < KSTEPS; ++st)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = Elem<T>::lo(qa[n][st][i]) * up, y = Elem<T>::hi(qa[n][st][i]) * up;
          const uint32_t high = pack_f16x2(x, y);
          const uint32_t low = pack_f16x2(x - Elem<__half>::lo(high), y - Elem<__half>::hi(high));
          qa[n][st][i] = kPair && (g & 1) ? low : high;
          if (!kPair) ql[kPair ? 0 : n][kPair ? 0 : st][i] = low;
        }
      // The scores' columns 2t (and 2t + 1) were loaded by lanes of row 2t (and 2t + 1).
      if (kPair) {
        qscale[0] = __shfl_sync(0xffffffffu, back, 8 * t);
      } else {
        qscale[NC > 1 ? 2 * n : 0] = __shfl_sync(0xffffffffu, back, 8 * t);
        qscale[NC > 1 ? 2 * n + 1 : 0] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
      }
    }
  }

  float acc[NG][VTILES][4];
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int j = 0; j < VTILES; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.0f;
  int erun[NC];  // biased exponents that the candidates' P are scaled to (fp16 products)
#pragma unroll
  for (int c = 0; c < NC; ++c) erun[c] = 30;

  const int krow_sw = KC >= 8 ? (g & 1) << 2 : 0;  // rows g and g + 8 alike
  int stage = 0;
  for (int n0 = 0; n0 < iters; ++n0) {
    copies_wait<S - 2>();
    if (wg > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + slice), "r"(32 * wg) : "memory");
    else __syncwarp();
    issue(n0 + S - 1, stage == 0 ? S - 1 : stage - 1);  // into the stage that the slice used last
    for (int j = 0; j < wg; ++j) {
      const int entry = (n0 * nslices + slice) * wg + j;
      if (entry >= entries || ncand == 0) break;
      const uint8_t* kt = paged_ring + (slice * S * wg + stage * wg + j) * Z::kStep;
      const uint8_t* vt = kt + kPagedTile * KROW;

      // Scores of keys g (values 0, 1 of a group) and g + 8 (2, 3), two sums
      // each, halves of a dependent chain.
      float s[2][NG][4];
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][n][e] = s[1][n][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        uint32_t kw[2][KB / 4];
        const int byte = i * 4 * KB + t * KB;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          load_piece<KB>(kt + (g + 8 * r) * KROW + ((byte >> 4) ^ krow_sw) * 16 + (byte & 15), kw[r]);
        constexpr int kPer = E4M3 ? KB / 4 : KB / 8;  // k = 16 steps of a piece
#pragma unroll
        for (int w = 0; w < kPer; ++w) {
          const int st = i * kPer + w;
          uint32_t a[4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            a[r] = E4M3 ? e4m3x2_to_f16x2(kw[r][E4M3 ? w : 0]) : kw[r][E4M3 ? 0 : 2 * w];
            a[2 + r] = E4M3 ? e4m3x2_hi_to_f16x2(kw[r][E4M3 ? w : 0]) : kw[r][E4M3 ? 0 : 2 * w + 1];
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            if (n >= groups) break;
            if (kSplitQ && !kPair) {
              mma16816<M>(s[0][n], a[0], a[1], a[2], a[3], qa[n][st][0], qa[n][st][1]);
              mma16816<M>(s[1][n], a[0], a[1], a[2], a[3], ql[kPair ? 0 : n][kSplitQ && !kPair ? st : 0][0],
                          ql[kPair ? 0 : n][kSplitQ && !kPair ? st : 0][1]);
            } else {
              mma16816<M>(s[st & 1][n], a[0], a[1], a[2], a[3], qa[n][st][0], qa[n][st][1]);
            }
          }
        }
      }

      // P of this lane's candidates at keys g and g + 8.
      const int key0 = paged_key(p, sp, entry);
      const bool part = p.func ? (sp.list[entry] & 0x8000) != 0 : key0 + kPagedTile > sp.k1;
      float ks[2], vs[2];
      if (E4M3) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          ks[r] = scale_value(vt[kPagedTile * VROW + g + 8 * r]);
          vs[r] = scale_value(vt[kPagedTile * VROW + 16 + g + 8 * r]);
        }
      }
      float pr[NC][2];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          pr[c][r] = 0.0f;
          if (c / 2 >= groups) continue;
          float x;
          if (kPair) {
            x = s[0][0][2 * r] + s[1][0][2 * r];
            if (kSplitQ) x += s[0][0][2 * r + 1] + s[1][0][2 * r + 1];
          } else {
            x = s[0][kPair ? 0 : c / 2][2 * r + (c & 1)] + s[1][kPair ? 0 : c / 2][2 * r + (c & 1)];
          }
          x *= qscale[c];
          if (E4M3) x *= ks[r];
          x = silu_exact(x);
          if (E4M3) x *= vs[r];
          pr[c][r] = x;
        }
      if (part) {
        // Interval by interval, all of this lane's candidates and keys at once.
        bool vis[NC][2];
#pragma unroll
        for (int c = 0; c < NC; ++c) vis[c][0] = vis[c][1] = false;
        if (p.func) {
          const int n = (p.nfunc + 1) / 2;
#pragma unroll 1
          for (int i = 0; i < n; ++i) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int cand = kPair ? t : c / 2 * 8 + 2 * t + (c & 1);
              const int* iv = sp.iv + (cg + (cand < ncand ? cand : 0)) * kPagedIv + 2 * i;
              const int lo = iv[0], hi = iv[1];
#pragma unroll
              for (int r = 0; r < 2; ++r) vis[c][r] |= lo <= key0 + g + 8 * r && key0 + g + 8 * r < hi;
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            vis[c][0] = key0 + g < sp.k1;
            vis[c][1] = key0 + g + 8 < sp.k1;
          }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r) pr[c][r] = vis[c][r] ? pr[c][r] : 0.0f;
      }
      if (kHalf) {
        // A candidate's scale follows the largest magnitude it has met.
        bool grow = false;
#pragma unroll
        for (int c = 0; c < NC; ++c)
          grow |= static_cast<int>(__float_as_uint(fmaxf(fabsf(pr[c][0]), fabsf(pr[c][1]))) >> 23) > erun[c];
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            float top = fmaxf(fabsf(pr[c][0]), fabsf(pr[c][1]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const int more = max(static_cast<int>(__float_as_uint(top) >> 23) - erun[c], 0);
            const float down = more < 127 ? __uint_as_float(static_cast<uint32_t>(127 - more) << 23) : 0.0f;
            erun[c] += more;
#pragma unroll
            for (int m = 0; m < VTILES; ++m)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (kPair || (e & 1) == (c & 1)) acc[kPair ? 0 : c / 2][m][e] *= down;
          }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float up = __uint_as_float(static_cast<uint32_t>(268 - erun[c]) << 23);  // below 2^15 at the largest
          pr[c][0] *= up;
          pr[c][1] *= up;
        }
      }
      // P^T operands: high and low parts in one (pair), or one each.
      uint32_t bh[NG][2], bl[NG][2];
      if (kPair) {
        const uint32_t h = Elem<M>::pack2(pr[0][0], pr[0][1]);
        bh[0][0] = transpose8(Elem<M>::pack2(pr[0][0], pr[0][0] - Elem<M>::lo(h)));
        bh[0][1] = transpose8(Elem<M>::pack2(pr[0][1], pr[0][1] - Elem<M>::hi(h)));
      } else {
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (n >= groups) break;
            const float x = pr[kPair ? 0 : 2 * n][r], y = pr[kPair ? 0 : 2 * n + 1][r];
            const uint32_t h = Elem<M>::pack2(x, y);
            bh[n][r] = transpose8(h);
            bl[n][r] = transpose8(Elem<M>::pack2(x - Elem<M>::lo(h), y - Elem<M>::hi(h)));
          }
      }

      // O^T += V^T P^T: rows g and g + 8 of a product are columns e and e + 1
      // of the lanes' pieces.
      const auto add = [&](int m, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          if (n >= groups) break;
          mma16816<M>(acc[n][m], a0, a1, a2, a3, bh[n][0], bh[n][1]);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          if (n >= groups) break;
          if (!kPair) mma16816<M>(acc[n][m], a0, a1, a2, a3, bl[n][0], bl[n][1]);
        }
      };
      if (E4M3) {
#pragma unroll
        for (int i = 0; i < VP; ++i) {
          uint32_t vw[4][VB / 4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + 8 * (r >> 1);
            const int byte = i * 8 * VB + g * VB;
            load_piece<VB>(vt + row * VROW + ((byte >> 4) ^ Z::v_swizzle(row)) * 16 + (byte & 15), vw[r]);
          }
#pragma unroll
          for (int w = 0; w < VB / 4; ++w) {
            // bytes (row 0, row 1) of columns 4w, 4w+1 and 4w+2, 4w+3
            const uint32_t x0 = __byte_perm(vw[0][w], vw[1][w], 0x5140);
            const uint32_t x1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
            const uint32_t y0 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
            const uint32_t y1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
            const int m = E4M3 ? i * VE / 2 + 2 * w : 0;
            add(m, e4m3x2_to_f16x2(x0), e4m3x2_hi_to_f16x2(x0), e4m3x2_to_f16x2(y0), e4m3x2_hi_to_f16x2(y0));
            add(E4M3 ? m + 1 : 0, e4m3x2_to_f16x2(x1), e4m3x2_hi_to_f16x2(x1), e4m3x2_to_f16x2(y1),
                e4m3x2_hi_to_f16x2(y1));
          }
        }
      } else {
        // Columns 16m .. 16m + 15 of the 16 rows, transposed on their way: lane
        // l gives row (l & 7) + 8 (l >> 4), columns 8 ((l >> 3) & 1) on.
        const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
        const uint32_t from = smem_u32(vt) + row * VROW;
#pragma unroll
        for (int m = 0; m < VTILES; ++m) {
          uint32_t v[4];
          load_transposed(from + ((2 * m + half) ^ Z::v_swizzle(row)) * 16, v);
          add(m, v[0], v[1], v[2], v[3]);
        }
      }
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }

  // This warp's sums.
  copies_wait<0>();
  __syncthreads();  // the ring is free: the sums take its place
  float* mine = sp.red + warp * ROWS * Z::kRedRow;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int r = kPair ? t : c / 2 * 8 + 2 * t + (c & 1);
    const float back = kHalf ? __uint_as_float(static_cast<uint32_t>(erun[c] - 14) << 23) : 1.0f;
    bool finite = true;
    if (r < ncand) {
      float* row = mine + r * Z::kRedRow;
#pragma unroll
      for (int m = 0; m < VTILES; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float(&a)[4] = acc[kPair ? 0 : c / 2][m];
          const float u = (kPair ? a[2 * e] + a[2 * e + 1] : a[2 * e + (c & 1)]) * back;
          finite = finite && fabsf(u) <= kMaxFinite;
          // 8-bit pages: column 2 (m % (VE / 2)) + e of this lane's piece m / (VE / 2)
          const int at = E4M3 ? (m / (VE / 2) * 8 + g) * Z::kBlock + m % (VE / 2) * 2 + e : 16 * m + 8 * e + g;
          row[at] = u;
        }
    }
    // A sum that is not finite may have met a value that its candidate does
    // not see (zero times infinity): those candidates are summed again, key by
    // key, over what they see alone.
    const uint32_t odd = __ballot_sync(0xffffffffu, !finite);
    if (odd != 0) __syncwarp();  // the lanes' stores above come before those of the second sum
    for (int l = 0; odd != 0 && l < 4; ++l) {
      if ((odd & (0x11111111u << l)) == 0) continue;
      const int again = kPair ? l : c / 2 * 8 + 2 * l + (c & 1);
      paged_scalar_sum<T, DQ, DV, E4M3, Z>(p, sp, cg + again, slice * wg, wg, entries, mine + again * Z::kRedRow);
    }
  }
  return wg;
}

// T: type of q, o and 16-bit pages. E4M3: 8-bit pages. MANY: any number of
// candidates, else one a sequence.
template <typename T, int DQ, int DV, bool E4M3, bool MANY, int W>
__global__ void __launch_bounds__(32 * W, PagedSizes<DQ, DV, E4M3, MANY, W>::kResident)
    paged_kernel(const PagedParams p) {
  using Z = PagedSizes<DQ, DV, E4M3, MANY, W>;
  __shared__ PagedTables<MANY> tables;

  chain();
  const int tid = threadIdx.x;
  const int64_t bid = blockIdx.x;
  // One candidate a sequence: first splits first, so that the last CTAs to start
  // are those of the sequences' ends, the shorter ones (8-bit pages, 256 users:
  // 118.9 us so, 120.4 us with a sequence's splits side by side). Splits that
  // follow the candidates take about the same time as they are, and are
  // better off side by side (67 us against 70).
  const int pairs = p.batch * p.cache.heads;
  const int split = static_cast<int>(MANY ? bid % p.nsplit : bid / pairs);
  const int bh = static_cast<int>(MANY ? bid / p.nsplit : bid % pairs);
  const int h = bh % p.cache.heads, b = bh / p.cache.heads;
  int cb = b, ce = b + 1;
  if (MANY) {
    cb = p.cand_offsets[b];
    ce = p.cand_offsets[b + 1];
  }
  const int keys = MANY ? paged_split_keys(p, ce - cb) : p.split;

  // A single candidate's intervals, read before the length is known.
  int raw[2 * kMaxIntervals - 1];
#pragma unroll
  for (int i = 0; i < 2 * kMaxIntervals - 1; ++i)
    raw[i] = !MANY && p.func && i < p.nfunc ? p.func[static_cast<int64_t>(i) * p.num_cand + b] : 0;

  PagedSplit sp;
  int splits;
  bool bad;
  if (!paged_open<MANY, Z::kThreads>(p, tables, b, h, split, cb, ce, keys, sp, splits, bad)) return;
  float* red = reinterpret_cast<float*>(paged_ring);
  sp.ring = smem_u32(paged_ring);
  sp.red = red;
  for (int c0 = cb; c0 < ce;) {
    sp.c0 = c0;
    int wg, rows;
    if (!MANY || ce - c0 <= 4) {
      wg = paged_pass<T, DQ, DV, E4M3, MANY, W, true>(p, sp, raw);
      rows = 4;
    } else {
      wg = paged_pass<T, DQ, DV, E4M3, MANY, W, !MANY>(p, sp, raw);
      rows = 16;
    }
    __syncthreads();
    // The slices' sums in slice order, four columns a thread.
    const int taken = min(ce - c0, wg * rows);
    for (int i = tid; i < taken * (DV / 4); i += Z::kThreads) {
      const int r = i / (DV / 4), d = i % (DV / 4) * 4;
      const float* from = red + r * Z::kRedRow + Z::red_column(d);  // warp r / rows of each slice
      float sum[4] = {from[0], from[1], from[2], from[3]};
      for (int w = wg; w < W; w += wg) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += from[w * rows * Z::kRedRow + e];
      }
      const int64_t at = static_cast<int64_t>(c0 + r) * p.cache.heads + h;
      if (splits > 1)
        *reinterpret_cast<float4*>(p.partial + (at * p.nsplit + split) * DV + d) =
            make_float4(sum[0], sum[1], sum[2], sum[3]);
      else if (!bad || p.zero)  // the sums of a bad sequence are zeros: it has no tiles
        *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * DV + d) =
            make_uint2(Elem<T>::pack2(sum[0] * p.inv_n, sum[1] * p.inv_n),
                       Elem<T>::pack2(sum[2] * p.inv_n, sum[3] * p.inv_n));
    }
    __syncthreads();
    c0 += taken;
  }
  if (splits > 1 && tid == 0) p.states[static_cast<int64_t>(bh) * p.nsplit + split] = bad ? 0 : 1;
}

// Joins the splits' sums of each (candidate, head), in a fixed order: WARPS
// warps take a share of the splits each, and their sums are added in warp
// order. Its blocks start while the last CTAs of paged_kernel run and wait for
// them. A sequence with one split was written there, and one with a bad split
// is left alone or becomes zeros, as are rows that no sequence is found for
// (offsets out of order).
template <typename T, int DV, int WARPS>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p) {
  chain();
  constexpr int kUnits = 8 / WARPS;  // (candidate, head) of a block
  __shared__ float4 red[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kUnits + warp / WARPS;
  const int64_t c = unit / p.cache.heads;
  const int h = static_cast<int>(unit - c * p.cache.heads);
  const bool row = c < p.num_cand;
  bool live = row, found = row;
  int b = static_cast<int>(c), first, keys = p.split;
  if (p.cand_offsets) {  // lanes of a warp ask for the same candidate
    found = find_sequence(p.cand_offsets, p.batch, row ? c : 0, b, first) && row;
    live = found && p.cand_offsets[0] == 0 && p.cand_offsets[p.batch] == p.num_cand &&
           p.cand_offsets[b + 1] <= p.num_cand;  // as paged_kernel has it
    keys = live ? paged_split_keys(p, p.cand_offsets[b + 1] - first) : p.split;
  }
  const int len = live ? p.lens[b] : 0;
  live = live && len > keys && len <= p.max_seqlen &&
         static_cast<int64_t>(len) <= (static_cast<int64_t>(p.max_pages) << p.cache.page_shift);
  const int splits = live ? (len + keys - 1) / keys : 0;
  const int32_t* states = p.states + (static_cast<int64_t>(b) * p.cache.heads + h) * p.nsplit;
  bool good = true;
  for (int s = lane; s < splits; s += 32) good = good && states[s] == 1;
  good = __all_sync(0xffffffffu, good);
  const bool blank = p.zero && row && (!found || (live && !good));
  live = good && live;

  const int share = (splits + WARPS - 1) / WARPS, s0 = warp % WARPS * share, s1 = min(splits, s0 + share);
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (live && lane < DV / 4) {
    const float4* from = reinterpret_cast<const float4*>(p.partial + unit * p.nsplit * DV) + lane;
#pragma unroll 8
    for (int s = s0; s < s1; ++s) {
      const float4 v = from[s * (DV / 4)];
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
  }
  if (WARPS > 1) {
    red[warp][lane] = sum;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      const float4 v = red[w][lane];
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
  }
  if ((live || blank) && lane < DV / 4)  // zeros where blank
    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + unit * DV + 4 * lane) =
        make_uint2(Elem<T>::pack2(sum.x * p.inv_n, sum.y * p.inv_n), Elem<T>::pack2(sum.z * p.inv_n, sum.w * p.inv_n));
}

cudaError_t launch_paged_bf16(const PagedParams& p, unsigned blocks, cudaStream_t stream);
cudaError_t launch_paged_f16(const PagedParams& p, unsigned blocks, cudaStream_t stream);
cudaError_t launch_paged_bf16_e4m3(const PagedParams& p, unsigned blocks, cudaStream_t stream);
cudaError_t launch_paged_f16_e4m3(const PagedParams& p, unsigned blocks, cudaStream_t stream);

}  // namespace hstu

// Candidate rows against a paged K/V cache where sequences have many of them: the
// kernel for bf16 and 8-bit pages with D_qk = D_v = 128, more than 16 candidates a
// sequence on average and N above 256 (paged_kernel takes the rest).
//
// The formula is paged.cuh's: o = sum_j silu(alpha q.k_j) / N v_j. With this many
// candidates paged_kernel is bound by its matrix instructions and the operands it
// brings into registers for each of its warps. Here the products run on
// tcgen05, transposed, so that the 128 keys of a step are the 128 rows of a product
// and the candidates its columns:
//   S^T (keys x cands)  = K Q^T       K and Q from shared memory
//   P = silu(alpha S), zero where not visible, in two 16-bit parts
//   O^T (Dv x cands)   += V^T [P_hi | P_lo]
// The sums of the two parts lie side by side in TMEM and are added at the end. Two
// bf16 parts leave a relative error of 2^-17 in P (fp32: 2^-24), against the
// output's rounding of 2^-8 (bf16) or 2^-11 (fp16). Thread r of a group of four
// warps has key r: its scores are one TMEM lane, its 8-bit scales two scalars, and
// its row of P one 128-byte row of shared memory, which is the layout that the
// second product reads P in (candidates along the row, keys down). A pass takes 64
// candidates, and each further pass reads the split's keys again.
//
// A step is eight 16-key tiles, listed as in paged_kernel: keys that no
// candidate sees are left out, and the second product skips tiles past the
// last. A CTA has eight warps: each copies one tile of a step, and two groups of four
// take 16 of 32 candidates each. K's next copy runs from the end of the first
// product on, V's from the end of the second, and two CTAs an SM (97 KB of shared
// memory, 256 columns of TMEM) fill each other's waits. (Warps of their own for
// copies, products and weights, two stages and one CTA an SM took 1.4 to 1.8 times
// as long: the first and last steps of a CTA then have nothing beside them.)
//
// 8-bit codes are exact in fp16 and in bf16. K is brought into the candidates'
// type, V and P into bf16, whose range is fp32's (P needs no scale there); fp16
// pages have no such exact form, which is why they are not taken here.
//
// Measured against paged_kernel, H = 4, 16-bit pages, us: 256 users of 1332 to 3994
// rows with 24 candidates each 256 (311), with 40 each 334 (533; the bytes alone take
// 206), 16 users of 20000 rows with 40 each 176 (294), 64 users of 512 to 2048 rows with
// 0 to 48 each 60 (64), with 16 each 49 (47). 8-bit pages: 40 each 405 (791), 0 to 48
// each 68 (85). With widths of 64, 0 to 48 each took 52 (45): a step's copies are
// too small there for its waits. 200 users with 8 to 48 each, N up to 304: 45 (55); N
// up to 176, a step or two a CTA, of which an SM holds two here and three there: 38 (34).
#pragma once

#include "paged.cuh"

namespace hstu {

constexpr int kManyDim = 128;  // D_qk and D_v

template <bool E4M3>
struct ManySizes {
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kKeys = kWarps * kPagedTile;  // of a step: the rows of a product
  static constexpr int kGroup = 32;                  // candidates of a second product
  static constexpr int ROW = kManyDim * (E4M3 ? 1 : 2);  // bytes of a cached row
  // Operands in blocks of 64 columns, 128 bytes a row, 16-byte pieces permuted by
  // row: K (2 blocks), V (2), P (1), Q (2).
  static constexpr int kBlock64 = kKeys * 128, kQBlock = kPagedPass * 128;
  static constexpr int kV = 2 * kBlock64, kP = 2 * kV, kQ = kP + kBlock64;
  static constexpr int kSmem = kQ + 2 * kQBlock + 1024;
  static constexpr int kTmem = 256;  // S: 64 columns, O: 64 for each of two groups
  static __device__ __forceinline__ int red_column(int d) { return d; }
};

// 32 lanes x 16 consecutive 32-bit TMEM columns; valid after tmem_ld16_wait.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// Writes to shared memory become visible to the products.
__device__ __forceinline__ void fence_operands() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void store16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Piece c (16 bytes) of row r of an operand in blocks of 64 columns.
template <int BLOCK>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  return (c >> 3) * BLOCK + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// One 16-key tile of k or of v, by one warp. 16-bit rows are
// copied asynchronously; 8-bit ones pass through registers, where they become M.
template <bool E4M3, typename M>
struct TileCopy {
  using Z = ManySizes<E4M3>;
  static constexpr int C = Z::ROW / 16, N = C / 2;  // pieces of a row, of a lane
  uint4 w[E4M3 ? N : 1];

  // rows at and past `nkeys` become zeros
  __device__ __forceinline__ void load(uint32_t dst, const void* base, int64_t row0, int nkeys, int lane) {
    const uint8_t* src = static_cast<const uint8_t*>(base) + row0 * Z::ROW + lane * 16;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = i * 32 + lane, r = u / C, c = u % C;
      if (E4M3)
        w[i] = r < nkeys ? *reinterpret_cast<const uint4*>(src + i * 512) : make_uint4(0, 0, 0, 0);
      else
        copy16(dst + piece_at<Z::kBlock64>(r, c), src + i * 512, r < nkeys);
    }
  }
  static __device__ __forceinline__ uint32_t pair(uint32_t f16x2) {
    return std::is_same<M, __half>::value ? f16x2 : pack_bf16x2(Elem<__half>::lo(f16x2), Elem<__half>::hi(f16x2));
  }
  // 8-bit rows: from registers into the operand.
  __device__ __forceinline__ void settle(uint32_t dst, int lane) {
    if constexpr (E4M3) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int u = i * 32 + lane, r = u / C, c = u % C;
        const uint4 x = w[i];
        const uint32_t words[4] = {x.x, x.y, x.z, x.w};
        uint32_t f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = pair(e4m3x2_to_f16x2(words[j]));
          f[2 * j + 1] = pair(e4m3x2_hi_to_f16x2(words[j]));
        }
        store16(dst + piece_at<Z::kBlock64>(r, 2 * c), f[0], f[1], f[2], f[3]);
        store16(dst + piece_at<Z::kBlock64>(r, 2 * c + 1), f[4], f[5], f[6], f[7]);
      }
    }
  }
};

template <typename T, bool E4M3>
__global__ void __launch_bounds__(256, 2) paged_many_kernel(const PagedParams p) {
  using Z = ManySizes<E4M3>;
  constexpr int DQ = kManyDim, DV = kManyDim;
  using PT = __nv_bfloat16;  // of V and P
  static_assert(E4M3 || std::is_same<T, PT>::value, "fp16 pages are not taken here");
  constexpr float kMaxFinite = 3.402823466e38f;
  __shared__ PagedTables<true> tables;
  __shared__ __align__(8) uint64_t bar_s, bar_o, bar_drain;
  __shared__ uint32_t tmem_base, odd[2];
  __shared__ int abort_word;

  chain();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bid = blockIdx.x;
  const int split = static_cast<int>(bid % p.nsplit), bh = static_cast<int>(bid / p.nsplit);
  const int h = bh % p.cache.heads, b = bh / p.cache.heads;
  const int cb = p.cand_offsets[b], ce = p.cand_offsets[b + 1];
  PagedSplit sp;
  int splits;
  bool bad;
  if (!paged_open<true, Z::kThreads>(p, tables, b, h, split, cb, ce, p.split, sp, splits, bad)) return;

  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(paged_ring) + 1023) & ~uintptr_t(1023));
  const uint32_t k_at = smem_u32(ring), v_at = k_at + Z::kV, p_at = k_at + Z::kP, q_at = k_at + Z::kQ;
  float* red = reinterpret_cast<float*>(ring);  // the sums of a pass, after its products
  const uint32_t s_bar = smem_u32(&bar_s), o_bar = smem_u32(&bar_o);
  volatile int* abort_flag = &abort_word;
  const int quarter = warp & 3, half = warp >> 2;
  const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
  const uint64_t dk = sdesc_sw128(k_at, 16, 1024), dq = sdesc_sw128(q_at, 16, 1024);
  const uint64_t dv = sdesc_sw128(v_at, Z::kBlock64, 1024), dp = sdesc_sw128(p_at, Z::kBlock64, 1024);
  constexpr uint32_t kIdescO = idesc_f16kind(128, 2 * Z::kGroup, true, true, Elem<PT>::kUmma);
  uint32_t s_phase = 0, o_phase = 0;
  bool ok = true;

  for (int c0 = cb; c0 < ce; c0 += kPagedPass) {
    sp.c0 = c0;
    const int total = min(ce - c0, kPagedPass);
    const int groups = total > Z::kGroup ? 2 : 1;
    const int raw[2 * kMaxIntervals - 1] = {};
    const int entries = p.func ? paged_list<true>(p, sp, total, raw) : sp.tiles;
    const int steps = (entries + Z::kWarps - 1) / Z::kWarps;

    // Row of the cache of this warp's tile in step t, and its keys.
    const auto tile_row = [&](int e, int& nkeys) {
      const int key0 = paged_key(p, sp, e);
      nkeys = sp.k1 - key0;
      return cache_row(p.cache, sp.pages[(key0 >> p.cache.page_shift) - sp.page0], sp.h,
                       key0 & ((1 << p.cache.page_shift) - 1));
    };
    TileCopy<E4M3, T> kc;
    TileCopy<E4M3, PT> vc;
    const uint32_t k_tile = k_at + warp * kPagedTile * 128, v_tile = v_at + warp * kPagedTile * 128;
    uint32_t kbyte = 0, vbyte = 0;  // scales of this thread's key in the step to come
    const auto fetch_k = [&](int t) {
      const int e = t * Z::kWarps + warp;
      if (e < entries) {
        int nkeys;
        const int64_t row = tile_row(e, nkeys);
        kc.load(k_tile, p.cache.k, row, nkeys, lane);
      }
      if (E4M3) {
        const int mine = t * Z::kWarps + 2 * quarter + (lane >> 4);
        if (mine < entries) {
          int nkeys;
          const int64_t row = tile_row(mine, nkeys) + (lane & 15);
          kbyte = p.cache.k_scale[row];
          vbyte = p.cache.v_scale[row];
        }
      } else {
        copies_commit();
      }
    };
    const auto fetch_v = [&](int t) {
      const int e = t * Z::kWarps + warp;
      if (e < entries) {
        int nkeys;
        const int64_t row = tile_row(e, nkeys);
        vc.load(v_tile, p.cache.v, row, nkeys, lane);
      }
      if (!E4M3) copies_commit();
    };
    fetch_k(0);
    fetch_v(0);

    for (int i = tid; i < total * (DQ / 8); i += Z::kThreads) {
      const int r = i / (DQ / 8), c = i % (DQ / 8);
      const T* qrow = static_cast<const T*>(p.q) + static_cast<int64_t>(c0 + r) * p.q_stride + static_cast<int64_t>(h) * DQ;
      const uint4 u = reinterpret_cast<const uint4*>(qrow)[c];
      store16(q_at + piece_at<Z::kQBlock>(r, c), u.x, u.y, u.z, u.w);
    }
    if (tid < 2) odd[tid] = 0;
    if (c0 == cb) {
      if (tid == 0) {
        abort_word = 0;
        mbar_init(s_bar, 1);
        mbar_init(o_bar, 1);
        mbar_init(smem_u32(&bar_drain), 1);
        fence_mbar_init();
      }
      if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_base), Z::kTmem);
        tmem_relinquish();
      }
    }

    for (int t = 0; t < steps; ++t) {
      if (E4M3) {
        if (t * Z::kWarps + warp < entries) kc.settle(k_tile, lane);
      } else {
        copies_wait<1>();
      }
      fence_operands();
      tc_fence_before();
      ok = __syncthreads_and(ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ts = *const_cast<volatile uint32_t*>(&tmem_base), to = ts + 2 * Z::kGroup;
      if (tid == 0) {
        const uint32_t idesc = idesc_f16kind(128, Z::kGroup * groups, false, false, Elem<T>::kUmma);
#pragma unroll
        for (int kk = 0; kk < DQ / 16; ++kk)
          umma_ss(ts, sdesc_advance(dk, (kk >> 2) * Z::kBlock64 + (kk & 3) * 32),
                  sdesc_advance(dq, (kk >> 2) * Z::kQBlock + (kk & 3) * 32), idesc, kk > 0);
        umma_commit(s_bar);
        // Only for a test, in the last pass: waits from here on give up, with a
        // product and copies in flight. (A wait with a condition or a limit of its
        // own cost 3 to 6%.)
        if (p.give_up && ce - c0 <= kPagedPass) *abort_flag = 1;
      }
      // This thread's key.
      const int mine = t * Z::kWarps + 2 * quarter + (lane >> 4);
      const float ks = E4M3 ? scale_value(kbyte) * p.alpha : p.alpha, vs = E4M3 ? scale_value(vbyte) : 1.0f;
      if (E4M3) {  // the next copies' registers are free as soon as the operands are written
        fetch_k(t + 1);
        if (t * Z::kWarps + warp < entries) vc.settle(v_tile, lane);
        fetch_v(t + 1);
      }
      int key = sp.k1;
      bool part = true;
      if (mine < entries) {
        const int key0 = paged_key(p, sp, mine);
        key = key0 + (lane & 15);
        part = p.func ? (sp.list[mine] & 0x8000) != 0 : key0 + kPagedTile > sp.k1;
      }
      ok = mbar_wait(s_bar, s_phase, abort_flag);
      s_phase ^= 1;
      tc_fence_after();
      if (!E4M3) fetch_k(t + 1);  // K is free
      for (int g = 0; g < groups; ++g) {
        const int first = g * Z::kGroup + 16 * half;  // candidates of this warp
        const bool busy = first < total && t * Z::kWarps + 2 * quarter < entries;
        uint32_t hi[8], lo[8];
        if (busy) {
          uint32_t s[16];
          __syncwarp();
          tmem_ld16(ts + lane_addr + first, s);
          tmem_ld16_wait(s);
          uint32_t seen = 0xffffu;
          if (part) {
            if (p.func) {
              seen = 0;
              const int n = (p.nfunc + 1) / 2;
#pragma unroll 1
              for (int i = 0; i < n; ++i)
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  const int* iv = sp.iv + min(first + c, total - 1) * kPagedIv + 2 * i;
                  seen |= (iv[0] <= key && key < iv[1] ? 1u : 0u) << c;
                }
            } else {
              seen = key < sp.k1 ? 0xffffu : 0u;
            }
          }
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            float x = silu_exact(__uint_as_float(s[c]) * ks), y = silu_exact(__uint_as_float(s[c + 1]) * ks);
            if (E4M3) {
              x *= vs;
              y *= vs;
            }
            x = (seen >> c) & 1u ? x : 0.0f;
            y = (seen >> (c + 1)) & 1u ? y : 0.0f;
            hi[c / 2] = Elem<PT>::pack2(x, y);
            lo[c / 2] = Elem<PT>::pack2(x - Elem<PT>::lo(hi[c / 2]), y - Elem<PT>::hi(hi[c / 2]));
          }
        }
        if (g > 0) {  // the first group's P has been read
          ok = mbar_wait(o_bar, o_phase, abort_flag) && ok;
          o_phase ^= 1;
        }
        if (busy) {
          const int r = 32 * quarter + lane;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            store16(p_at + piece_at<Z::kBlock64>(r, 2 * half + c), hi[4 * c], hi[4 * c + 1], hi[4 * c + 2],
                    hi[4 * c + 3]);
            store16(p_at + piece_at<Z::kBlock64>(r, 4 + 2 * half + c), lo[4 * c], lo[4 * c + 1], lo[4 * c + 2],
                    lo[4 * c + 3]);
          }
        }
        if (g == 0 && !E4M3) copies_wait<1>();  // V has arrived
        fence_operands();
        tc_fence_before();
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (tid == 0) {
          tc_fence_after();
          const int tiles = min(Z::kWarps, entries - t * Z::kWarps);
          for (int kk = 0; kk < tiles; ++kk)
            umma_ss(to + g * 2 * Z::kGroup, sdesc_advance(dv, kk * kPagedTile * 128),
                    sdesc_advance(dp, kk * kPagedTile * 128), kIdescO, t > 0 || kk > 0);
          umma_commit(o_bar);
        }
      }
      if (!ok) break;
      ok = mbar_wait(o_bar, o_phase, abort_flag);
      o_phase ^= 1;
      if (!E4M3) fetch_v(t + 1);  // V is free
    }
    if (!E4M3) copies_wait<0>();
    ok = __syncthreads_and(ok && (steps == 0 || *abort_flag == 0));
    if (!ok) break;

    // The sums: column c of O^T and its second part.
    tc_fence_after();
    if (steps == 0) {
      for (int i = tid; i < total * DV; i += Z::kThreads) red[i] = 0.0f;
    } else {
      const uint32_t to = *const_cast<volatile uint32_t*>(&tmem_base) + 2 * Z::kGroup;
      for (int g = 0; g < groups; ++g) {
        const int first = g * Z::kGroup + 16 * half;
        if (first >= total) break;
        uint32_t x[16], y[16];
        tmem_ld16(to + lane_addr + g * 2 * Z::kGroup + 16 * half, x);
        tmem_ld16(to + lane_addr + g * 2 * Z::kGroup + Z::kGroup + 16 * half, y);
        tmem_ld16_wait(x);
        tmem_ld16_wait(y);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          if (first + c >= total) break;
          const float u = __uint_as_float(x[c]) + __uint_as_float(y[c]);
          red[(first + c) * DV + 32 * quarter + lane] = u;
          if (!(fabsf(u) <= kMaxFinite)) atomicOr(odd + g, 1u << (16 * half + c));
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    // Sums that are not finite may have met what their candidate does not see.
    if ((odd[0] | odd[1]) != 0) {
      for (int r = warp; r < total; r += Z::kWarps)
        if ((odd[r >> 5] >> (r & 31)) & 1u)
          paged_scalar_sum<T, DQ, DV, E4M3, Z>(p, sp, r, 0, Z::kWarps, entries, red + r * DV);
      __syncthreads();
    }
    for (int i = tid; i < total * (DV / 4); i += Z::kThreads) {
      const int r = i / (DV / 4), d = i % (DV / 4) * 4;
      const float4 sum = *reinterpret_cast<const float4*>(red + r * DV + d);
      const int64_t at = static_cast<int64_t>(c0 + r) * p.cache.heads + h;
      if (splits > 1)
        *reinterpret_cast<float4*>(p.partial + (at * p.nsplit + split) * DV + d) = sum;
      else if (!bad || p.zero)
        *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * DV + d) =
            make_uint2(Elem<T>::pack2(sum.x * p.inv_n, sum.y * p.inv_n),
                       Elem<T>::pack2(sum.z * p.inv_n, sum.w * p.inv_n));
    }
    __syncthreads();  // the sums' place and Q are free
  }

  if (!ok) {  // a product did not end in time: leave none in flight
    if (p.zero && splits == 1) paged_zero_rows(p.o, p.cache.heads, DV, sp.h, sp.c0, sp.ce);
    if (!E4M3) copies_wait<0>();
    if (tid == 0) {
      umma_commit(smem_u32(&bar_drain));
      mbar_wait_drain(smem_u32(&bar_drain), 0);
      if (p.header) atomicOr(p.header + kHdrErr, kErrTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(*const_cast<volatile uint32_t*>(&tmem_base), Z::kTmem);
  }
  if (splits > 1 && tid == 0) p.states[static_cast<int64_t>(bh) * p.nsplit + split] = ok && !bad ? 1 : 0;
}

// Launches the kernel for the widths of p.cache (one function for each type,
// in a translation unit of its own so that they compile in parallel).
template <typename T, bool E4M3, int DQ, int DV, bool MANY, int W>
cudaError_t launch_paged_one(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  constexpr int kSmem = PagedSizes<DQ, DV, E4M3, MANY, W>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(paged_kernel<T, DQ, DV, E4M3, MANY, W>, kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(paged_kernel<T, DQ, DV, E4M3, MANY, W>, dim3(blocks), 32 * W, kSmem, stream, p);
}

template <typename T, bool E4M3>
cudaError_t launch_paged_many(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  using Z = ManySizes<E4M3>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = ensure_smem_limit(paged_many_kernel<T, E4M3>, Z::kSmem, done);
  if (e != cudaSuccess) return e;
  return launch_chained(paged_many_kernel<T, E4M3>, dim3(blocks), Z::kThreads, Z::kSmem, stream, p);
}

template <typename T, int DV, int WARPS>
cudaError_t launch_paged_join(const PagedParams& p, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(p.num_cand) * p.cache.heads;
  const dim3 grid(static_cast<unsigned>((units + 8 / WARPS - 1) / (8 / WARPS)));
  return launch_chained(paged_join_kernel<T, DV, WARPS>, grid, 256, 0, stream, p);
}
template <typename T, bool E4M3, int DQ, int DV>
cudaError_t launch_paged_widths(const PagedParams& p, unsigned blocks, cudaStream_t stream) {
  // Eight warps a CTA where there is at most a CTA for each of 152 SMs: each warp
  // has half the tiles to go through. (One row for each of 8 users of 700 to 1400
  // rows: 7.2 us so, 8.2 us with four. With 200 to 256 CTAs it made no
  // difference or cost 2%; 128 keys are two tiles a warp either way.)
  const bool wide = blocks <= 152u && p.max_seqlen > 128;
  cudaError_t e = cudaSuccess;
  if (!p.cand_offsets) {
    e = wide ? launch_paged_one<T, E4M3, DQ, DV, false, kPagedWarpsWide>(p, blocks, stream)
             : launch_paged_one<T, E4M3, DQ, DV, false, kPagedWarps>(p, blocks, stream);
  } else if (!p.tensor) {
    e = launch_paged_one<T, E4M3, DQ, DV, true, kPagedWarps>(p, blocks, stream);
  } else {
    if constexpr (DQ == kManyDim && DV == kManyDim && (E4M3 || !std::is_same<T, __half>::value))
      e = launch_paged_many<T, E4M3>(p, blocks, stream);
    else
      e = cudaErrorInvalidValue;  // paged_layout asks for it with those alone
  }
  if (e != cudaSuccess || p.nsplit == 1 || p.num_cand == 0) return e;
  // A warp for each (candidate, head), or a block where those are few.
  if (static_cast<int64_t>(p.num_cand) * p.cache.heads <= 1216) return launch_paged_join<T, DV, 8>(p, stream);
  return launch_paged_join<T, DV, 1>(p, stream);
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

}  // namespace hstu

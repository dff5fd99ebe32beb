// Writing rows into the paged K/V cache and reading them back.
//
// Both kernels move each row once. A thread holds one slot (16 columns) of
// one (row, head) of k or of v; the threads of a row are neighbours in a
// warp, so that a row's largest magnitude, which sets the scale of its 8-bit
// codes, is a few shuffles away. The blocks of the k rows come first in the
// grid, those of the v rows after them.
#include "cache.cuh"
#include "rope.cuh"

namespace hstu {

constexpr int kCacheThreads = 256;

struct CacheParams {
  CacheView cache;
  void* k;  // jagged rows: written into the cache, or read back
  void* v;
  int64_t k_stride, v_stride;
  const int32_t* seq_offsets;
  const int32_t* starts;  // position of each sequence's first row; null: 0
  const int32_t* page_table;
  const int32_t* positions;  // for the rotation; null: the row's position
  const uint64_t* turns;     // null: k is not rotated
  int32_t* header;           // null: skipped rows are not reported
  int64_t rows, k_blocks;
  int32_t batch, max_pages, rotary;
  float magnitude;
};

// Page-table lookup of jagged row t: its position and its (page, slot).
// False (and the error word set) where the row has no valid place.
__device__ __forceinline__ bool place_row(const CacheParams& p, int64_t t, int64_t& pos, int64_t& page, int& slot) {
  int b, first;
  bool ok = find_sequence(p.seq_offsets, p.batch, t, b, first);
  if (ok) {
    const int start = p.starts ? __ldg(p.starts + b) : 0;
    pos = t - first + start;
    ok = start >= 0 && pos < (static_cast<int64_t>(p.max_pages) << p.cache.page_shift);
  }
  if (ok) {
    page = __ldg(p.page_table + static_cast<int64_t>(b) * p.max_pages + (pos >> p.cache.page_shift));
    slot = static_cast<int>(pos & ((1 << p.cache.page_shift) - 1));
    ok = page >= 0 && page < p.cache.num_pages;
  }
  if (!ok && p.header) atomicOr(p.header + kHdrErr, kErrInput);
  return ok;
}

// Block 0 also checks the ends and the order of seq_offsets, where there is
// an error word to report to.
__device__ __forceinline__ void check_offsets(const CacheParams& p) {
  if (!p.header || blockIdx.x != 0) return;
  bool bad = p.seq_offsets[0] != 0 || static_cast<int64_t>(p.seq_offsets[p.batch]) != p.rows;
  for (int b = threadIdx.x; b < p.batch; b += kCacheThreads) bad |= p.seq_offsets[b] > p.seq_offsets[b + 1];
  if (bad) atomicOr(p.header + kHdrErr, kErrInput);
}

// The unit (row, head, slot) of this thread in the k or v part of the grid.
struct CacheUnit {
  int64_t row;
  int head, slot, width;
  bool is_v, live;
};
__device__ __forceinline__ CacheUnit cache_unit(const CacheParams& p) {
  CacheUnit u;
  u.is_v = blockIdx.x >= p.k_blocks;
  u.width = u.is_v ? p.cache.dim_v : p.cache.dim;
  const int slots = u.width / 16;
  const int64_t unit =
      (static_cast<int64_t>(blockIdx.x) - (u.is_v ? p.k_blocks : 0)) * kCacheThreads + threadIdx.x;
  u.slot = static_cast<int>(unit) & (slots - 1);
  const int64_t rh = unit / slots;
  u.row = rh / p.cache.heads;
  u.head = static_cast<int>(rh - u.row * p.cache.heads);
  u.live = u.row < p.rows;
  return u;
}

// ROPE: 0 none, 1 half layout, 2 interleaved.
template <typename T, bool E4M3, int ROPE>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
  check_offsets(p);
  const CacheUnit u = cache_unit(p);
  int64_t pos = 0, page = 0;
  int slot_in_page = 0;
  const bool ok = u.live && place_row(p, u.row, pos, page, slot_in_page);
  const bool turned = ROPE != 0 && !u.is_v && 16 * u.slot < p.rotary;
  int c0 = 16 * u.slot, c1 = c0 + 8;
  if (ROPE != 0 && !u.is_v) slot_columns(u.slot, p.rotary, ROPE == 2, c0, c1);
  uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
  if (ok) {
    const T* row = static_cast<const T*>(u.is_v ? p.v : p.k) + u.row * (u.is_v ? p.v_stride : p.k_stride) +
                   static_cast<int64_t>(u.head) * u.width;
    u0 = *reinterpret_cast<const uint4*>(row + c0);
    u1 = *reinterpret_cast<const uint4*>(row + c1);
  }
  float a[8], b[8];
  if (E4M3 || turned) {
    unpack8<T>(u0, a);
    unpack8<T>(u1, b);
  }
  if (turned && ok) {
    float c[8], s[8];
    rope_factors(p.turns, 8 * u.slot, p.positions ? __ldg(p.positions + u.row) : pos, p.magnitude,
                 1.0f, c, s);
    rotate_pairs<ROPE == 2>(a, b, c, s);
  }
  const int64_t at = ok ? cache_row(p.cache, page, u.head, slot_in_page) : 0;
  if (!E4M3) {
    if (!ok) return;
    if (turned) {
      u0 = pack8<T>(a);
      u1 = pack8<T>(b);
    }
    T* out = static_cast<T*>(u.is_v ? p.cache.v : p.cache.k) + at * u.width;
    *reinterpret_cast<uint4*>(out + c0) = u0;
    *reinterpret_cast<uint4*>(out + c1) = u1;
    return;
  }
  // Largest finite magnitude of the row: this thread's 16 values, then the
  // row's 2, 4 or 8 threads.
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = fabsf(a[i]), y = fabsf(b[i]);
    top = fmaxf(top, x <= 3.402823466e38f ? x : 0.0f);
    top = fmaxf(top, y <= 3.402823466e38f ? y : 0.0f);
  }
  const int slots = u.width / 16;
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, top, off);
    if (off < slots) top = fmaxf(top, o);
  }
  if (!ok) return;
  const uint32_t byte = scale_byte(top);
  const float inv = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte), exact
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = fabsf(a[i]) <= 3.402823466e38f ? a[i] * inv : __uint_as_float(0x7fc00000u);
    b[i] = fabsf(b[i]) <= 3.402823466e38f ? b[i] * inv : __uint_as_float(0x7fc00000u);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = e4m3x2(a[4 * i], a[4 * i + 1]) | (e4m3x2(a[4 * i + 2], a[4 * i + 3]) << 16);
    w[2 + i] = e4m3x2(b[4 * i], b[4 * i + 1]) | (e4m3x2(b[4 * i + 2], b[4 * i + 3]) << 16);
  }
  uint8_t* out = static_cast<uint8_t*>(u.is_v ? p.cache.v : p.cache.k) + at * u.width;
  if (c1 == c0 + 8) {
    *reinterpret_cast<uint4*>(out + c0) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(out + c0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(out + c1) = make_uint2(w[2], w[3]);
  }
  if (u.slot == 0) (u.is_v ? p.cache.v_scale : p.cache.k_scale)[at] = static_cast<uint8_t>(byte);
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
  check_offsets(p);
  const CacheUnit u = cache_unit(p);
  if (!u.live) return;
  int64_t pos, page;
  int slot_in_page;
  if (!place_row(p, u.row, pos, page, slot_in_page)) return;
  const int64_t at = cache_row(p.cache, page, u.head, slot_in_page);
  T* out = static_cast<T*>(u.is_v ? p.v : p.k) + (u.row * p.cache.heads + u.head) * u.width + 16 * u.slot;
  const void* base = u.is_v ? p.cache.v : p.cache.k;
  uint4 u0, u1;
  if (E4M3) {
    const uint4 codes =
        __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at * u.width + 16 * u.slot));
    const float scale = scale_value(__ldg((u.is_v ? p.cache.v_scale : p.cache.k_scale) + at));
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = e4m3x2_to_f16x2(w[i / 2] >> (16 * (i & 1)));
      f[2 * i] = Elem<__half>::lo(h) * scale;
      f[2 * i + 1] = Elem<__half>::hi(h) * scale;
    }
    u0 = make_uint4(Elem<T>::pack2(f[0], f[1]), Elem<T>::pack2(f[2], f[3]), Elem<T>::pack2(f[4], f[5]),
                    Elem<T>::pack2(f[6], f[7]));
    u1 = make_uint4(Elem<T>::pack2(f[8], f[9]), Elem<T>::pack2(f[10], f[11]), Elem<T>::pack2(f[12], f[13]),
                    Elem<T>::pack2(f[14], f[15]));
  } else {
    const T* in = static_cast<const T*>(base) + at * u.width + 16 * u.slot;
    u0 = __ldg(reinterpret_cast<const uint4*>(in));
    u1 = __ldg(reinterpret_cast<const uint4*>(in) + 1);
  }
  *reinterpret_cast<uint4*>(out) = u0;
  *reinterpret_cast<uint4*>(out + 8) = u1;
}

static hstu_status_t cache_common(const hstu_cache_t* cache, const int32_t* seq_offsets, int32_t batch, int64_t rows,
                                  const int32_t* starts, const int32_t* page_table, int32_t max_pages, void* ws,
                                  size_t ws_bytes, CacheParams* p, int64_t* blocks) {
  *p = CacheParams{};
  const hstu_status_t st = check_cache(cache, &p->cache);
  if (st != HSTU_OK) return st;
  if (batch < 1 || rows < 0 || rows > INT32_MAX || max_pages < 1) return HSTU_ERR_INVALID_ARG;
  const auto bad4 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 != 0; };
  if (!seq_offsets || !page_table || bad4(seq_offsets) || bad4(starts) || bad4(page_table))
    return HSTU_ERR_INVALID_ARG;
  if (ws && (reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < kHdrWords * 4)) return HSTU_ERR_WORKSPACE;
  const auto blocks_of = [&](int width) {
    return (rows * p->cache.heads * (width / 16) + kCacheThreads - 1) / kCacheThreads;
  };
  p->k_blocks = blocks_of(p->cache.dim);
  *blocks = p->k_blocks + blocks_of(p->cache.dim_v);
  if (*blocks > INT32_MAX) return HSTU_ERR_UNSUPPORTED;
  p->seq_offsets = seq_offsets;
  p->starts = starts;
  p->page_table = page_table;
  p->header = static_cast<int32_t*>(ws);
  p->rows = rows;
  p->batch = batch;
  p->max_pages = max_pages;
  return HSTU_OK;
}

static cudaError_t clear_header(void* ws, cudaStream_t stream) {
  return ws ? cudaMemsetAsync(ws, 0, kHdrWords * 4, stream) : cudaSuccess;
}

template <typename T, bool E4M3>
static void launch_write(const CacheParams& p, unsigned blocks, int rope, cudaStream_t stream) {
  if (rope == 0) cache_write_kernel<T, E4M3, 0><<<blocks, kCacheThreads, 0, stream>>>(p);
  else if (rope == 1) cache_write_kernel<T, E4M3, 1><<<blocks, kCacheThreads, 0, stream>>>(p);
  else cache_write_kernel<T, E4M3, 2><<<blocks, kCacheThreads, 0, stream>>>(p);
}

template <typename T>
static void launch_write_typed(const CacheParams& p, unsigned blocks, bool e4m3, int rope, cudaStream_t stream) {
  if (e4m3) launch_write<T, true>(p, blocks, rope, stream);
  else launch_write<T, false>(p, blocks, rope, stream);
}

template <typename T>
static void launch_read_typed(const CacheParams& p, unsigned blocks, bool e4m3, cudaStream_t stream) {
  if (e4m3) cache_read_kernel<T, true><<<blocks, kCacheThreads, 0, stream>>>(p);
  else cache_read_kernel<T, false><<<blocks, kCacheThreads, 0, stream>>>(p);
}

}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_attn_cache_write(const hstu_cache_t* cache, const void* k, int64_t k_stride,
                                             const void* v, int64_t v_stride, const int32_t* seq_offsets,
                                             int32_t batch, int64_t rows, const int32_t* cache_lens,
                                             const int32_t* page_table, int32_t max_pages, const hstu_rope_t* rope,
                                             const int32_t* positions, void* ws, size_t ws_bytes, void* stream) {
  hstu::CacheParams p;
  int64_t blocks = 0;
  hstu_status_t st =
      hstu::cache_common(cache, seq_offsets, batch, rows, cache_lens, page_table, max_pages, ws, ws_bytes, &p, &blocks);
  if (st != HSTU_OK) return st;
  if (!cache_lens || reinterpret_cast<uintptr_t>(positions) % 4 != 0 || (positions && !rope))
    return HSTU_ERR_INVALID_ARG;
  if (rows > 0 && (!hstu::rows_ok(k, k_stride, p.cache.heads, p.cache.dim) ||
                   !hstu::rows_ok(v, v_stride, p.cache.heads, p.cache.dim_v)))
    return HSTU_ERR_INVALID_ARG;
  if (rope) {
    st = hstu::check_rope(rope, p.cache.dim);
    if (st != HSTU_OK) return st;
    p.turns = rope->turns;
    p.rotary = rope->rotary_dim;
    p.magnitude = rope->magnitude;
  }
  p.k = const_cast<void*>(k);
  p.v = const_cast<void*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (hstu::clear_header(ws, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  if (rows == 0) return HSTU_OK;
  const int mode = rope ? (rope->interleaved ? 2 : 1) : 0;
  if (cache->dtype == HSTU_DTYPE_F16)
    hstu::launch_write_typed<__half>(p, static_cast<unsigned>(blocks), cache->e4m3 != 0, mode, cs);
  else
    hstu::launch_write_typed<__nv_bfloat16>(p, static_cast<unsigned>(blocks), cache->e4m3 != 0, mode, cs);
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API hstu_status_t hstu_attn_cache_read(const hstu_cache_t* cache, void* k, void* v, const int32_t* seq_offsets,
                                            int32_t batch, int64_t rows, const int32_t* starts,
                                            const int32_t* page_table, int32_t max_pages, void* ws, size_t ws_bytes,
                                            void* stream) {
  hstu::CacheParams p;
  int64_t blocks = 0;
  const hstu_status_t st =
      hstu::cache_common(cache, seq_offsets, batch, rows, starts, page_table, max_pages, ws, ws_bytes, &p, &blocks);
  if (st != HSTU_OK) return st;
  const auto bad = [](const void* q) { return !q || reinterpret_cast<uintptr_t>(q) % 16 != 0; };
  if (rows > 0 && (bad(k) || bad(v))) return HSTU_ERR_INVALID_ARG;
  p.k = k;
  p.v = v;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (hstu::clear_header(ws, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  if (rows == 0) return HSTU_OK;
  if (cache->dtype == HSTU_DTYPE_F16)
    hstu::launch_read_typed<__half>(p, static_cast<unsigned>(blocks), cache->e4m3 != 0, cs);
  else
    hstu::launch_read_typed<__nv_bfloat16>(p, static_cast<unsigned>(blocks), cache->e4m3 != 0, cs);
  return cudaGetLastError() == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"

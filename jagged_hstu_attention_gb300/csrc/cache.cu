// Writing rows into the paged K/V cache and reading them back.
//
// Both kernels move each row once. A thread holds one slot (two 8-column
// chunks) of the k and v rows of one token, for several heads: the token's
// sequence, its page and the slot's cosines and sines are found once for all
// of them. The threads of a row are neighbours in a warp, so that a row's
// largest magnitude, which sets the scale of its 8-bit codes, is a few
// shuffles away.
//
// Bound by memory: 86000 rows (4 heads of 128) into 16-bit pages, k rotated, take
// 56 us, 6.2 TB/s; with a thread for each (row, head, slot), which searched its
// sequence and computed its cosines alone, they took 100 us. A chunk of 3500 rows
// into 8-bit pages and 90000 rows read back from them take 50 us, 5.7 TB/s, of
// which the read is 43 us.
#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "rope.cuh"

namespace hstu {

// Threads of a block. (86000 rows written take 56 us with 128 threads and 58
// us with 256, whose registers leave an SM two blocks; 90000 rows read back take
// 2 us less with 256.)
constexpr int kWriteThreads = 128, kReadThreads = 256;
constexpr int kCacheHeads = 4;  // heads of a thread where there are rows enough to fill the GPU

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
  int64_t rows;
  int32_t batch, max_pages, rotary;
  int32_t slots;  // threads of a token: those of the wider of k and v
  bool one_head;  // heads of a thread: 1 or kCacheHeads
  bool zero;      // reader: skipped rows become zeros
  float magnitude;
};

// Page-table lookup of jagged row t: its position and its (page, slot).
// False (and the error word set) where the row has no valid place. Every lane
// of the warp calls it; rows past the last are nobody's and search as the last.
__device__ __forceinline__ bool place_row(const CacheParams& p, int64_t t, int64_t& pos, int64_t& page, int& slot) {
  int b, first;
  bool ok = find_sequence(p.seq_offsets, p.batch, min(t, p.rows - 1), b, first);
  if (t >= p.rows) return false;
  if (ok) {
    const int start = p.starts ? p.starts[b] : 0;
    pos = t - first + start;
    ok = start >= 0 && pos < (static_cast<int64_t>(p.max_pages) << p.cache.page_shift);
  }
  if (ok) {
    page = p.page_table[static_cast<int64_t>(b) * p.max_pages + (pos >> p.cache.page_shift)];
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
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x) bad |= p.seq_offsets[b] > p.seq_offsets[b + 1];
  if (bad) atomicOr(p.header + kHdrErr, kErrInput);
}

// One head's 16 columns, in registers.
struct Chunks {
  uint4 a, b;
};
template <typename T>
__device__ __forceinline__ Chunks load_chunks(const T* row, const SlotColumns& k) {
  return Chunks{*reinterpret_cast<const uint4*>(row + k.c0), *reinterpret_cast<const uint4*>(row + k.c1)};
}

// Writes one head's slot into the cache at row `at` of `out`. Every thread of
// the row calls it; those without a part of it (`live` false) only take part
// in the shuffles.
template <typename T, bool E4M3, int ROPE>
__device__ __forceinline__ void write_chunks(Chunks u, const SlotColumns& k, bool turned, const float (&c)[8],
                                             const float (&s)[8], bool live, int slots, void* out, uint8_t* scales,
                                             int64_t at, int width, bool first) {
  float a[8], b[8];
  if (E4M3 || ROPE != 0) {
    unpack8<T>(u.a, a);
    unpack8<T>(u.b, b);
  }
  if (ROPE != 0 && turned) rotate_pairs<ROPE == 2>(a, b, c, s);
  if (!E4M3) {
    if (!live) return;
    if (ROPE != 0 && turned) u = Chunks{pack8<T>(a), pack8<T>(b)};
    T* row = static_cast<T*>(out) + at * width;
    *reinterpret_cast<uint4*>(row + k.c0) = u.a;
    *reinterpret_cast<uint4*>(row + k.c1) = u.b;
    return;
  }
  // Largest finite magnitude of the row: this thread's 16 values, then the
  // row's 2, 4 or 8 threads.
  constexpr float kMaxFinite = 3.402823466e38f;
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = fabsf(a[i]), y = fabsf(b[i]);
    top = fmaxf(top, x <= kMaxFinite ? x : 0.0f);
    top = fmaxf(top, y <= kMaxFinite ? y : 0.0f);
  }
  if (!live) top = 0.0f;
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, top, off);
    if (off < slots) top = fmaxf(top, o);
  }
  if (!live) return;
  const uint32_t byte = scale_byte(top);
  const float inv = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte), exact
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = fabsf(a[i]) <= kMaxFinite ? a[i] * inv : __uint_as_float(0x7fc00000u);
    b[i] = fabsf(b[i]) <= kMaxFinite ? b[i] * inv : __uint_as_float(0x7fc00000u);
  }
  uint8_t* row = static_cast<uint8_t*>(out) + at * width;
  *reinterpret_cast<uint2*>(row + k.c0) = make_uint2(e4m3x2(a[0], a[1]) | (e4m3x2(a[2], a[3]) << 16),
                                                     e4m3x2(a[4], a[5]) | (e4m3x2(a[6], a[7]) << 16));
  *reinterpret_cast<uint2*>(row + k.c1) = make_uint2(e4m3x2(b[0], b[1]) | (e4m3x2(b[2], b[3]) << 16),
                                                     e4m3x2(b[4], b[5]) | (e4m3x2(b[6], b[7]) << 16));
  if (first) scales[at] = static_cast<uint8_t>(byte);
}

// ROPE: 0 none, 1 half layout, 2 interleaved.
template <typename T, bool E4M3, int ROPE, int HEADS>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const CacheParams p) {
  chain();
  check_offsets(p);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int slot = static_cast<int>(unit) & (p.slots - 1);
  const int64_t row = unit / p.slots;
  const int h0 = blockIdx.y * HEADS, heads = min(HEADS, p.cache.heads - h0);
  const bool in = row < p.rows;
  const bool has_k = in && 16 * slot < p.cache.dim, has_v = in && 16 * slot < p.cache.dim_v;
  const SlotColumns kc = slot_columns(slot, p.cache.dim, ROPE != 0 ? p.rotary : 0, ROPE == 2);
  const SlotColumns vc = slot_columns(slot, p.cache.dim_v, 0, false);
  // The rows' loads do not wait for the search of their place.
  const T* krow = static_cast<const T*>(p.k) + row * p.k_stride + static_cast<int64_t>(h0) * p.cache.dim;
  const T* vrow = static_cast<const T*>(p.v) + row * p.v_stride + static_cast<int64_t>(h0) * p.cache.dim_v;
  Chunks ku[HEADS], vu[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    ku[i] = vu[i] = Chunks{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (i >= heads) continue;
    if (has_k) ku[i] = load_chunks(krow + i * p.cache.dim, kc);
    if (has_v) vu[i] = load_chunks(vrow + i * p.cache.dim_v, vc);
  }
  int64_t pos = 0, page = 0;
  int slot_in_page = 0;
  const bool ok = place_row(p, row, pos, page, slot_in_page);
  float c[8], s[8];
  const bool turned = ROPE != 0 && has_k && kc.turned;
  if (turned && ok)
    rope_factors(p.turns, kc.first, kc.second, p.positions ? p.positions[row] : pos, p.magnitude, 1.0f, c, s);
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    if (i >= heads) break;
    const int64_t at = cache_row(p.cache, page, h0 + i, slot_in_page);
    write_chunks<T, E4M3, ROPE>(ku[i], kc, turned && ok, c, s, ok && has_k, p.cache.dim / 16, p.cache.k,
                                p.cache.k_scale, at, p.cache.dim, slot == 0);
    write_chunks<T, E4M3, 0>(vu[i], vc, false, c, s, ok && has_v, p.cache.dim_v / 16, p.cache.v, p.cache.v_scale, at,
                             p.cache.dim_v, slot == 0);
  }
}

// x cut to [-top, top]; NaN stays.
__device__ __forceinline__ float cut(float x, float top) {
  float r;
  asm("{\n\t.reg .f32 low;\n\tmax.NaN.f32 low, %1, %3;\n\tmin.NaN.f32 %0, low, %2;\n\t}"
      : "=f"(r)
      : "f"(x), "f"(top), "f"(-top));
  return r;
}

// Eight codes times their scale, rounded to T. The largest values of T may have
// been rounded up to a code above them (fp16: 63488 and up to 65536): those come
// back as T's largest, not as infinity.
template <typename T>
__device__ __forceinline__ uint4 decode8(const uint2 codes, float scale) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? codes.y : codes.x;
    const uint32_t lo = e4m3x2_to_f16x2(w), hi = e4m3x2_hi_to_f16x2(w);
    f[4 * i] = Elem<__half>::lo(lo) * scale;
    f[4 * i + 1] = Elem<__half>::hi(lo) * scale;
    f[4 * i + 2] = Elem<__half>::lo(hi) * scale;
    f[4 * i + 3] = Elem<__half>::hi(hi) * scale;
  }
  constexpr float kTop = std::is_same<T, __half>::value ? 65504.0f : 3.38953139e38f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = cut(f[i], kTop);
  return pack8<T>(f);
}

// A skipped row's slot, 16 columns of the row that begins at `at`.
template <typename T>
__device__ __forceinline__ void zero_slot(void* out, int64_t at, int slot, int width) {
  if (16 * slot >= width) return;
  uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(out) + at + 16 * slot);
  to[0] = to[1] = make_uint4(0, 0, 0, 0);
}

template <typename T, bool E4M3, int HEADS>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const CacheParams p) {
  chain();
  check_offsets(p);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int slot = static_cast<int>(unit) & (p.slots - 1);
  const int64_t row = unit / p.slots;
  const int h0 = blockIdx.y * HEADS, heads = min(HEADS, p.cache.heads - h0);
  int64_t pos, page;
  int slot_in_page;
  if (!place_row(p, row, pos, page, slot_in_page)) {
    if (p.zero && row < p.rows) {
      for (int i = 0; i < heads; ++i) {
        zero_slot<T>(p.k, (row * p.cache.heads + h0 + i) * p.cache.dim, slot, p.cache.dim);
        zero_slot<T>(p.v, (row * p.cache.heads + h0 + i) * p.cache.dim_v, slot, p.cache.dim_v);
      }
    }
    return;
  }
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    const int width = part ? p.cache.dim_v : p.cache.dim;
    if (16 * slot >= width) continue;
    const SlotColumns k = slot_columns(slot, width, 0, false);
    const void* base = part ? p.cache.v : p.cache.k;
    const uint8_t* scales = part ? p.cache.v_scale : p.cache.k_scale;
    T* out = static_cast<T*>(part ? p.v : p.k) + (row * p.cache.heads + h0) * width;
    Chunks u[HEADS];
    uint32_t byte[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      if (i >= heads) break;
      const int64_t at = cache_row(p.cache, page, h0 + i, slot_in_page);
      if (E4M3) {
        const uint8_t* codes = static_cast<const uint8_t*>(base) + at * width;
        const uint2 x = *reinterpret_cast<const uint2*>(codes + k.c0);
        const uint2 y = *reinterpret_cast<const uint2*>(codes + k.c1);
        u[i].a = make_uint4(x.x, x.y, y.x, y.y);
        byte[i] = scales[at];
      } else {
        u[i] = load_chunks(static_cast<const T*>(base) + at * width, k);
      }
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      if (i >= heads) break;
      if (E4M3) {
        const float scale = scale_value(byte[i]);
        u[i].b = decode8<T>(make_uint2(u[i].a.z, u[i].a.w), scale);
        u[i].a = decode8<T>(make_uint2(u[i].a.x, u[i].a.y), scale);
      }
      *reinterpret_cast<uint4*>(out + i * width + k.c0) = u[i].a;
      *reinterpret_cast<uint4*>(out + i * width + k.c1) = u[i].b;
    }
  }
}

static hstu_status_t cache_common(const hstu_cache_t* cache, const int32_t* seq_offsets, int32_t batch, int64_t rows,
                                  const int32_t* starts, const int32_t* page_table, int32_t max_pages, void* ws,
                                  size_t ws_bytes, int threads, CacheParams* p, dim3* grid) {
  *p = CacheParams{};
  const hstu_status_t st = check_cache(cache, &p->cache);
  if (st != HSTU_OK) return st;
  if (batch < 1 || rows < 0 || rows > INT32_MAX || max_pages < 1) return HSTU_ERR_INVALID_ARG;
  const auto bad4 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 != 0; };
  if (!seq_offsets || !page_table || bad4(seq_offsets) || bad4(starts) || bad4(page_table))
    return HSTU_ERR_INVALID_ARG;
  if (ws && (reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < kHdrWords * 4)) return HSTU_ERR_WORKSPACE;
  p->slots = (p->cache.dim > p->cache.dim_v ? p->cache.dim : p->cache.dim_v) / 16;
  const int64_t blocks = (rows * p->slots + threads - 1) / threads;
  // A thread for each head while that does not fill the GPU (1024 threads on each
  // of 152 SMs): the heads of a call with few rows are then moved at once.
  p->one_head = blocks * p->cache.heads * threads <= 152 * 1024;
  *grid = dim3(static_cast<unsigned>(blocks > 0 ? blocks : 1),
               p->one_head ? p->cache.heads : (p->cache.heads + kCacheHeads - 1) / kCacheHeads);
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

template <typename T, bool E4M3, int HEADS>
static cudaError_t launch_write(const CacheParams& p, dim3 grid, int rope, cudaStream_t stream) {
  void (*kernel)(CacheParams) = rope == 0   ? cache_write_kernel<T, E4M3, 0, HEADS>
                                : rope == 1 ? cache_write_kernel<T, E4M3, 1, HEADS>
                                            : cache_write_kernel<T, E4M3, 2, HEADS>;
  return launch_chained(kernel, grid, kWriteThreads, 0, stream, p);
}

template <typename T>
static cudaError_t launch_write_typed(const CacheParams& p, dim3 grid, bool e4m3, int rope, cudaStream_t stream) {
  if (p.one_head)
    return e4m3 ? launch_write<T, true, 1>(p, grid, rope, stream) : launch_write<T, false, 1>(p, grid, rope, stream);
  return e4m3 ? launch_write<T, true, kCacheHeads>(p, grid, rope, stream)
              : launch_write<T, false, kCacheHeads>(p, grid, rope, stream);
}

template <typename T>
static cudaError_t launch_read_typed(const CacheParams& p, dim3 grid, bool e4m3, cudaStream_t stream) {
  void (*kernel)(CacheParams) =
      p.one_head ? (e4m3 ? cache_read_kernel<T, true, 1> : cache_read_kernel<T, false, 1>)
                 : (e4m3 ? cache_read_kernel<T, true, kCacheHeads> : cache_read_kernel<T, false, kCacheHeads>);
  return launch_chained(kernel, grid, kReadThreads, 0, stream, p);
}

static hstu_status_t cache_read(const hstu_cache_t* cache, void* k, void* v, const int32_t* seq_offsets, int32_t batch,
                                int64_t rows, const int32_t* starts, const int32_t* page_table, int32_t max_pages,
                                void* ws, size_t ws_bytes, bool zero, cudaStream_t stream) {
  CacheParams p;
  dim3 grid;
  const hstu_status_t st = cache_common(cache, seq_offsets, batch, rows, starts, page_table, max_pages, ws, ws_bytes,
                                        kReadThreads, &p, &grid);
  if (st != HSTU_OK) return st;
  const auto bad = [](const void* q) { return !q || reinterpret_cast<uintptr_t>(q) % 16 != 0; };
  if (rows > 0 && (bad(k) || bad(v))) return HSTU_ERR_INVALID_ARG;
  const int64_t k_row = 2ll * p.cache.heads * p.cache.dim, v_row = 2ll * p.cache.heads * p.cache.dim_v;
  if (rows_meet(k, k_row, k_row, v, v_row, v_row, rows)) return HSTU_ERR_INVALID_ARG;
  p.k = k;
  p.v = v;
  p.zero = zero;
  if (clear_header(ws, stream) != cudaSuccess) return HSTU_ERR_CUDA;
  if (rows == 0 && !ws) return HSTU_OK;  // with an error word, the offsets are checked all the same
  const cudaError_t e = cache->dtype == HSTU_DTYPE_F16
                            ? launch_read_typed<__half>(p, grid, cache->e4m3 != 0, stream)
                            : launch_read_typed<__nv_bfloat16>(p, grid, cache->e4m3 != 0, stream);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_attn_cache_write(const hstu_cache_t* cache, const void* k, int64_t k_stride,
                                             const void* v, int64_t v_stride, const int32_t* seq_offsets,
                                             int32_t batch, int64_t rows, const int32_t* cache_lens,
                                             const int32_t* page_table, int32_t max_pages, const hstu_rope_t* rope,
                                             const int32_t* positions, void* ws, size_t ws_bytes, void* stream) {
  hstu::CacheParams p;
  dim3 grid;
  hstu_status_t st =
      hstu::cache_common(cache, seq_offsets, batch, rows, cache_lens, page_table, max_pages, ws, ws_bytes,
                         hstu::kWriteThreads, &p, &grid);
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
  if (rows == 0 && !ws) return HSTU_OK;  // with an error word, the offsets are checked all the same
  const int mode = rope ? (rope->interleaved ? 2 : 1) : 0;
  const cudaError_t e = cache->dtype == HSTU_DTYPE_F16
                            ? hstu::launch_write_typed<__half>(p, grid, cache->e4m3 != 0, mode, cs)
                            : hstu::launch_write_typed<__nv_bfloat16>(p, grid, cache->e4m3 != 0, mode, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API hstu_status_t hstu_attn_cache_read(const hstu_cache_t* cache, void* k, void* v, const int32_t* seq_offsets,
                                            int32_t batch, int64_t rows, const int32_t* starts,
                                            const int32_t* page_table, int32_t max_pages, void* ws, size_t ws_bytes,
                                            void* stream) {
  return hstu::cache_read(cache, k, v, seq_offsets, batch, rows, starts, page_table, max_pages, ws, ws_bytes, false,
                          static_cast<cudaStream_t>(stream));
}

HSTU_API hstu_status_t hstu_attn_cache_read_zeroed(const hstu_cache_t* cache, void* k, void* v,
                                                   const int32_t* seq_offsets, int32_t batch, int64_t rows,
                                                   const int32_t* starts, const int32_t* page_table,
                                                   int32_t max_pages, void* ws, size_t ws_bytes, void* stream) {
  return hstu::cache_read(cache, k, v, seq_offsets, batch, rows, starts, page_table, max_pages, ws, ws_bytes, true,
                          static_cast<cudaStream_t>(stream));
}

}  // extern "C"

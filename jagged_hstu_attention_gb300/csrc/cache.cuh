// The paged K/V cache on the device: where a row lies, and the 8-bit codes.
#pragma once

#include "../../include/hstu_attn.h"
#include "common.cuh"

namespace hstu {

// Fields of hstu_cache_t that the kernels use.
struct CacheView {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t num_pages;
  int32_t page_shift;  // log2 of the page size
  int32_t heads, dim, dim_v;
};

// Row index (in rows of one head) of `slot` of (page, head).
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int64_t page, int head, int slot) {
  return ((page * c.heads + head) << c.page_shift) + slot;
}

// The sequence of jagged row t, the last b with offsets[b] <= t; false where
// the offsets do not bracket t. The rows of a warp are neighbours: the warp
// finds the sequence of its first row together, 32 offsets a step, and each
// lane goes on from there: four sequences one by one, which is where the rows of
// a step lie, then in steps that double and halve again, so that a run of
// empty sequences costs two loads for each doubling of its length. (A search by
// halving from the start takes 6 to 10 dependent loads, most of the time of a
// call with few rows.) Every lane of the warp calls it, those without a row of
// their own with a row of the batch.
__device__ __forceinline__ bool find_sequence(const int32_t* offsets, int batch, int64_t t, int& b, int& first) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = __shfl_sync(0xffffffffu, t, 0);
  int lo = 0, n = batch;
  while (n > 1) {
    const int step = (n - 1) / 32 + 1, at = lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, at < n && offsets[lo + at] <= t0);
    const int k = max(31 - __clz(below), 0);  // the last probe at or below t0
    lo += k * step;
    n = min(step, n - k * step);
  }
  b = lo;
  first = offsets[b];
  int next = offsets[b + 1];
  for (int i = 0; i < 4 && next <= t && b + 1 < batch; ++i) {
    ++b;
    first = next;
    next = offsets[b + 1];
  }
  if (next <= t && b + 1 < batch) {
    uint32_t step = 1, end = b + 1;  // offsets[end] <= t so far
    while (end < batch && offsets[end] <= t) {
      b = end;
      step *= 2;
      end = b + min(step, batch - b);
    }
    while (end - b > 1) {
      const int mid = b + (end - b) / 2;
      if (offsets[mid] <= t) b = mid;
      else end = mid;
    }
    first = offsets[b];
    next = offsets[b + 1];
  }
  return first >= 0 && first <= t && t < next;
}

// 2^(byte - 127); 2^-127 is below the normal numbers, hence the maximum.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(max(byte << 23, 0x00400000u));
}

// Scale byte of a row whose largest finite magnitude is `top`: the smallest
// power of two 2^e with top <= 448 * 2^e. With top = m 2^E, 1 <= m < 2, and
// 448 = 1.75 * 2^8 that is e = E - 8, or E - 7 where m > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float top) {
  const uint32_t u = __float_as_uint(top);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// Two floats to 8-bit codes (round to nearest even), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// The low two codes of w as fp16 (exact), the lower one in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}

// The high two codes of w.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Host checks of a cache; fills the kernels' view of it.
inline hstu_status_t check_cache(const hstu_cache_t* c, CacheView* out) {
  if (!c) return HSTU_ERR_INVALID_ARG;
  const int dv = c->head_dim_v != 0 ? c->head_dim_v : c->head_dim;
  const auto width_ok = [](int d) { return d == 32 || d == 64 || d == 128; };
  if (!width_ok(c->head_dim) || !width_ok(dv)) return HSTU_ERR_UNSUPPORTED;
  if (c->dtype != HSTU_DTYPE_BF16 && c->dtype != HSTU_DTYPE_F16) return HSTU_ERR_UNSUPPORTED;
  int shift = 0;
  while (shift < 9 && (1 << shift) != c->page_size) ++shift;
  if (shift < 4 || shift > 8) return HSTU_ERR_UNSUPPORTED;
  if (c->num_heads < 1 || c->num_heads > 65535) return c->num_heads < 1 ? HSTU_ERR_INVALID_ARG : HSTU_ERR_UNSUPPORTED;
  if (c->num_pages < 1 || c->num_pages > INT32_MAX || (c->e4m3 != 0 && c->e4m3 != 1)) return HSTU_ERR_INVALID_ARG;
  const auto bad = [](const void* p) { return !p || reinterpret_cast<uintptr_t>(p) % 16 != 0; };
  if (bad(c->k) || bad(c->v) || (c->e4m3 && (bad(c->k_scale) || bad(c->v_scale)))) return HSTU_ERR_INVALID_ARG;
  *out = CacheView{c->k,     c->v,         c->k_scale,    c->v_scale, c->num_pages,
                   shift,    c->num_heads, c->head_dim,   dv};
  return HSTU_OK;
}

}  // namespace hstu

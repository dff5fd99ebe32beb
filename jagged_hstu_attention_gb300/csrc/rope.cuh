// Rotary positions on the device: exact phases, sine and cosine of a phase,
// and the rotation of 8 pairs (shared by the rotation kernel and the cache
// writer, which rotates k on its way into the pages).
#pragma once

#include <algorithm>

#include "../../include/hstu_attn.h"
#include "common.cuh"

namespace hstu {

// cos and sin of `phase` / 2^32 turns. The nearest quarter turn leaves an
// angle x in [-pi/4, pi/4], where the Taylor series to x^10 (cos) and x^9
// (sin) are within 2e-9 of the functions, below the rounding of fp32.
__device__ __forceinline__ void phase_cos_sin(uint32_t phase, float& c, float& s) {
  const uint32_t quarter = (phase + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(phase - (quarter << 30))) * 1.46291807926715968e-9f;
  const float x2 = x * x;
  float sn = fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, -1/7!
  sn = fmaf(x2, sn, 8.33333333e-3f);                     // 1/5!
  sn = fmaf(x2, sn, -1.66666667e-1f);                    // -1/3!
  sn = fmaf(x * x2, sn, x);
  float cs = fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);  // -1/10!, 1/8!
  cs = fmaf(x2, cs, -1.38888889e-3f);                    // -1/6!
  cs = fmaf(x2, cs, 4.16666667e-2f);                     // 1/4!
  cs = fmaf(x2, cs, -0.5f);
  cs = fmaf(x2, cs, 1.0f);
  // quarter 0: (c, s); 1: (-s, c); 2: (-c, -s); 3: (s, -c)
  const bool swap = quarter & 1u;
  const float a = swap ? sn : cs, b = swap ? cs : sn;
  c = ((quarter + 1u) & 2u) ? -a : a;
  s = (quarter & 2u) ? -b : b;
}

// m cos and m sin of pairs first .. first + 3 and second .. second + 3 at
// position pos; sign = -1 for the transposed rotation. pos * turns wraps modulo
// one turn in 64-bit integers, so the phase is exact at any position, negative
// ones included.
__device__ __forceinline__ void rope_factors(const uint64_t* turns, int first, int second, int64_t pos, float magnitude,
                                             float sign, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t phase = static_cast<uint64_t>(pos) * turns[i < 4 ? first + i : second + i - 4];
    phase_cos_sin(static_cast<uint32_t>(phase >> 32), c[i], s[i]);
    c[i] *= magnitude;
    s[i] *= magnitude * sign;
  }
}

// Rotates the 8 pairs held in two 8-column chunks: (a[i], b[i]) in the half
// layout; (a[2i], a[2i+1]), then (b[2i], b[2i+1]) in the interleaved one.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_pairs(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& x = INTERLEAVED ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
    float& y = INTERLEAVED ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
    const float u = x * c[i] - y * s[i];
    y = y * c[i] + x * s[i];
    x = u;
  }
}

// A row of `width` columns, the first `rotary` of them rotated, is dealt to
// width / 16 slots of two 8-column chunks: those of the rotated columns first.
// The chunks lie half of their part apart, so that the slots' neighbouring
// 16-byte loads and stores fill whole sectors, and the half layout finds both
// members of its pairs.
struct SlotColumns {
  int c0, c1;         // columns of the chunks
  int first, second;  // pairs of the factors (rotated slots)
  bool turned;
};
__device__ __forceinline__ SlotColumns slot_columns(int slot, int width, int rotary, bool interleaved) {
  SlotColumns k;
  k.turned = 16 * slot < rotary;
  const int base = k.turned ? 0 : rotary, part = k.turned ? rotary : width - rotary;
  k.c0 = base + 8 * (slot - base / 16);
  k.c1 = k.c0 + part / 2;
  k.first = interleaved ? k.c0 / 2 : k.c0;
  k.second = interleaved ? k.c1 / 2 : k.c0 + 4;
  return k;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = Elem<T>::lo(w[i]);
    f[2 * i + 1] = Elem<T>::hi(w[i]);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(Elem<T>::pack2(f[0], f[1]), Elem<T>::pack2(f[2], f[3]), Elem<T>::pack2(f[4], f[5]),
                    Elem<T>::pack2(f[6], f[7]));
}

// Host check of a rotation against a head of `dim` columns.
inline hstu_status_t check_rope(const hstu_rope_t* r, int dim) {
  if (!r || !r->turns || reinterpret_cast<uintptr_t>(r->turns) % 8 != 0) return HSTU_ERR_INVALID_ARG;
  if (r->rotary_dim < 16 || r->rotary_dim % 16 != 0 || r->rotary_dim > dim) return HSTU_ERR_UNSUPPORTED;
  if (r->interleaved != 0 && r->interleaved != 1) return HSTU_ERR_INVALID_ARG;
  if (!(r->magnitude == r->magnitude)) return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

// Host check of a (rows, H, dim) tensor with rows `stride` elements apart.
inline bool rows_ok(const void* p, int64_t stride, int heads, int dim) {
  return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride >= static_cast<int64_t>(heads) * dim &&
         stride % 8 == 0;
}

// Whether one of n rows of `wa` bytes, `sa` bytes apart from a on, shares memory
// with one of n rows of b. (The rows of two slices of one projection lie
// between each other without meeting.)
inline bool rows_meet(const void* a, int64_t sa, int64_t wa, const void* b, int64_t sb, int64_t wb, int64_t n) {
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  if (n <= 0 || d >= (n - 1) * sa + wa || -d >= (n - 1) * sb + wb) return false;
  const auto floor_div = [](int64_t x, int64_t y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
  // Rows of b, of which row j begins at d + j sb, that meet [x, x + wa): -wb < d + j sb - x < wa.
  const auto first = [&](int64_t x) { return floor_div(x - d - wb, sb) + 1; };
  const auto last = [&](int64_t x) { return floor_div(x - d + wa - 1, sb); };
  if (sa == sb)  // the same for every row of a, but for the ends
    return std::max(first(0), 1 - n) <= std::min(last(0), n - 1);
  for (int64_t i = 0; i < n; ++i)
    if (std::max<int64_t>(first(i * sa), 0) <= std::min(last(i * sa), n - 1)) return true;
  return false;
}

inline bool head_width_ok(int d) { return d == 32 || d == 64 || d == 128; }

}  // namespace hstu

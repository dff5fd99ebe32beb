// Shared pieces of the layer's row operators (embedding rows, norms, products
// with an epilogue): element types, 8-column chunks and host checks.
#pragma once

#include "../../include/hstu_attn.h"
#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace hstu {

// Eight consecutive columns of a row in 32 bits. (fp32 as one access of 32 bytes, a
// whole sector: two of 16, each of every other half sector of a warp's, write at half
// the rate, 4.1 against 7.6 TB/s.)
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
               : "l"(p)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  unpack8<T>(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = pack8<T>(f);
}

inline bool row_dtype_ok(int dtype) { return dtype == HSTU_DTYPE_BF16 || dtype == HSTU_DTYPE_F16; }
inline bool aligned_to(const void* p, uintptr_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }

// Whether two ranges of memory share a byte.
inline bool ranges_meet(const void* a, int64_t bytes_a, const void* b, int64_t bytes_b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && bytes_a > 0 && bytes_b > 0 && x < y + static_cast<uint64_t>(bytes_b) &&
         y < x + static_cast<uint64_t>(bytes_a);
}

// `n` rows of `width` bytes, `stride` bytes apart; p may be null.
struct RowSpan {
  const void* p;
  int64_t stride, width, n;
};
inline bool spans_meet(const RowSpan& a, const RowSpan& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0) return false;
  if (a.n == b.n && a.n > 1) return rows_meet(a.p, a.stride, a.width, b.p, b.stride, b.width, a.n);
  return ranges_meet(a.p, (a.n - 1) * a.stride + a.width, b.p, (b.n - 1) * b.stride + b.width);
}
// Whether an output shares memory with an input or another output.
template <int I, int O>
bool outputs_meet(const RowSpan (&in)[I], const RowSpan (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (spans_meet(in[i], out[o])) return true;
    for (int i = 0; i < o; ++i)
      if (spans_meet(out[i], out[o])) return true;
  }
  return false;
}

}  // namespace hstu

// fp32 arithmetic on register pairs: one instruction for two values, which is what
// row kernels that are short of issue slots want (the rate of the pipe is the same).
#pragma once

#include "sm103_primitives.cuh"

namespace hstu {

__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void pair_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t pair_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pair_bits(uint32_t lo, uint32_t hi) {
  return pair_of(__uint_as_float(lo), __uint_as_float(hi));
}
template <typename T>
__device__ __forceinline__ uint64_t unpack_pair(uint32_t w) {
  return pair_of(Elem<T>::lo(w), Elem<T>::hi(w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
  float a, b;
  pair_split(v, a, b);
  return Elem<T>::pack2(a, b);
}

}  // namespace hstu

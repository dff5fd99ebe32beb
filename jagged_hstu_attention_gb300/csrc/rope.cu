// Rotary positions: rotates q and k by the positions of their rows, forward
// and (transposed) backward. The attention kernels take no positional bias,
// so this is how positions reach the scores.
//
// Each row of q and k is read and written once. A thread holds one slot (8
// pairs, or 16 columns that are copied) of one token: it computes the slot's
// cosines and sines once, in registers, and applies them to the heads of q
// and k in turn. Nothing is read from a table of positions: the phase of a
// position is one 64-bit integer product, and about 25 instructions a pair give
// its cosine and sine.
//
// Bound by memory: q and k of 81920 tokens (4 heads of 128), forward and
// backward, take 101.5 us, 6.6 TB/s, 97% of a plain copy; 32749 tokens of 8 heads
// in fp16, half of each head rotated, read from rows four times as long, 42 us
// (6.4 TB/s). A step of 64 tokens takes 2.2 us, about the time of an empty launch.
#include <cmath>

#include "internal.h"
#include "rope.cuh"

namespace hstu {

constexpr int kRopeThreads = 128;
constexpr int kRopeHeads = 4;  // heads of a thread where there are tokens enough to fill the GPU

struct RopeParams {
  const void* in[2];
  void* out[2];
  int64_t in_stride[2], out_stride[2];
  const int32_t* positions;
  const uint64_t* turns;
  int64_t tokens;
  int32_t heads, tensors, rotary;
  float magnitude, sign;
};

template <typename T, int D, int HPT, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  chain();
  constexpr int kSlots = D / 16;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int64_t token = unit / kSlots;
  const int slot = static_cast<int>(unit % kSlots);
  if (token >= p.tokens) return;
  const SlotColumns k = slot_columns(slot, D, p.rotary, INTERLEAVED);
  float c[8], s[8];
  if (k.turned) rope_factors(p.turns, k.first, k.second, p.positions[token], p.magnitude, p.sign, c, s);
  const int h0 = blockIdx.y * HPT;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if (t >= p.tensors) break;
    const T* in = static_cast<const T*>(p.in[t]) + token * p.in_stride[t];
    T* out = static_cast<T*>(p.out[t]) + token * p.out_stride[t];
    uint4 u0[HPT], u1[HPT];
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      if (h0 + i >= p.heads) break;
      u0[i] = *reinterpret_cast<const uint4*>(in + (h0 + i) * D + k.c0);
      u1[i] = *reinterpret_cast<const uint4*>(in + (h0 + i) * D + k.c1);
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      if (h0 + i >= p.heads) break;
      if (k.turned) {
        float a[8], b[8];
        unpack8<T>(u0[i], a);
        unpack8<T>(u1[i], b);
        rotate_pairs<INTERLEAVED>(a, b, c, s);
        u0[i] = pack8<T>(a);
        u1[i] = pack8<T>(b);
      }
      *reinterpret_cast<uint4*>(out + (h0 + i) * D + k.c0) = u0[i];
      *reinterpret_cast<uint4*>(out + (h0 + i) * D + k.c1) = u1[i];
    }
  }
}

template <typename T, int D, int HPT>
static cudaError_t launch_rope(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  const int64_t blocks = (p.tokens * (D / 16) + kRopeThreads - 1) / kRopeThreads;
  const dim3 grid(static_cast<unsigned>(blocks), (p.heads + HPT - 1) / HPT);
  return launch_chained(interleaved ? rope_kernel<T, D, HPT, true> : rope_kernel<T, D, HPT, false>, grid, kRopeThreads,
                        0, stream, p);
}

template <typename T, int D>
static cudaError_t launch_rope_heads(const RopeParams& p, bool interleaved, cudaStream_t stream) {
  // A thread for each head while that does not fill the GPU (1024 threads on each
  // of 152 SMs).
  const int64_t blocks = (p.tokens * (D / 16) + kRopeThreads - 1) / kRopeThreads;
  if (blocks * p.heads * kRopeThreads <= 152 * 1024) return launch_rope<T, D, 1>(p, interleaved, stream);
  return launch_rope<T, D, kRopeHeads>(p, interleaved, stream);
}

template <typename T>
static cudaError_t launch_rope_typed(const RopeParams& p, int dim, bool interleaved, cudaStream_t stream) {
  if (dim == 128) return launch_rope_heads<T, 128>(p, interleaved, stream);
  if (dim == 64) return launch_rope_heads<T, 64>(p, interleaved, stream);
  return launch_rope_heads<T, 32>(p, interleaved, stream);
}

}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_attn_rope_table(const hstu_rope_spec_t* spec, uint64_t* turns, float* magnitude) {
  if (!spec || !turns || !magnitude) return HSTU_ERR_INVALID_ARG;
  const int R = spec->rotary_dim;
  if (R < 16 || R > 128 || R % 16 != 0) return HSTU_ERR_UNSUPPORTED;
  if (spec->scaling < HSTU_ROPE_NONE || spec->scaling > HSTU_ROPE_YARN) return HSTU_ERR_UNSUPPORTED;
  if (!(spec->base > 1.0) || !std::isfinite(spec->base)) return HSTU_ERR_INVALID_ARG;
  const bool scaled = spec->scaling != HSTU_ROPE_NONE;
  if (scaled && (!(spec->factor >= 1.0) || !std::isfinite(spec->factor))) return HSTU_ERR_INVALID_ARG;
  const bool yarn = spec->scaling == HSTU_ROPE_YARN;
  if (yarn && (!(spec->original_len >= 1.0) || !std::isfinite(spec->original_len) || !(spec->slow_turns > 0.0) ||
               !(spec->fast_turns > spec->slow_turns) || !std::isfinite(spec->fast_turns)))
    return HSTU_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  const double base = spec->scaling == HSTU_ROPE_NTK
                          ? spec->base * std::pow(spec->factor, static_cast<double>(R) / (R - 2))
                          : spec->base;
  if (!std::isfinite(base)) return HSTU_ERR_INVALID_ARG;
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(base, -2.0 * i / R);
    if (spec->scaling == HSTU_ROPE_LINEAR) f /= spec->factor;
    if (yarn) {
      double keep = (spec->original_len * f / kTwoPi - spec->slow_turns) / (spec->fast_turns - spec->slow_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      f *= keep + (1.0 - keep) / spec->factor;
    }
    // f <= 1 radian, so below a sixth of a turn: the fraction fits 64 bits.
    turns[i] = static_cast<uint64_t>(std::ldexp(f / kTwoPi, 64));
  }
  *magnitude = yarn ? static_cast<float>(0.1 * std::log(spec->factor) + 1.0) : 1.0f;
  return HSTU_OK;
}

HSTU_API hstu_status_t hstu_attn_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                                      int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                      const int32_t* positions, int64_t tokens, int32_t num_heads, int32_t head_dim,
                                      int32_t dtype, const hstu_rope_t* rope, int32_t backward, void* stream) {
  if (tokens < 0 || tokens > INT32_MAX || num_heads < 1) return HSTU_ERR_INVALID_ARG;
  if (!hstu::head_width_ok(head_dim) || num_heads > 65535) return HSTU_ERR_UNSUPPORTED;
  if (dtype != HSTU_DTYPE_BF16 && dtype != HSTU_DTYPE_F16) return HSTU_ERR_UNSUPPORTED;
  const hstu_status_t st = hstu::check_rope(rope, head_dim);
  if (st != HSTU_OK) return st;
  if (tokens == 0) return HSTU_OK;
  if (!hstu::rows_ok(q, q_stride, num_heads, head_dim) || !hstu::rows_ok(q_out, q_out_stride, num_heads, head_dim) ||
      (k && (!hstu::rows_ok(k, k_stride, num_heads, head_dim) ||
             !hstu::rows_ok(k_out, k_out_stride, num_heads, head_dim))) ||
      !positions || reinterpret_cast<uintptr_t>(positions) % 4 != 0)
    return HSTU_ERR_INVALID_ARG;
  if ((q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride))
    return HSTU_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(num_heads) * head_dim * 2;
  const auto meet = [&](const void* a, int64_t sa, const void* b, int64_t sb) {
    return hstu::rows_meet(a, 2 * sa, row, b, 2 * sb, row, tokens);
  };
  if (q_out != q && meet(q_out, q_out_stride, q, q_stride)) return HSTU_ERR_INVALID_ARG;
  if (k && ((k_out != k && meet(k_out, k_out_stride, k, k_stride)) || meet(q_out, q_out_stride, k, k_stride) ||
            meet(k_out, k_out_stride, q, q_stride) || meet(q_out, q_out_stride, k_out, k_out_stride)))
    return HSTU_ERR_INVALID_ARG;
  hstu::RopeParams p{};
  p.in[0] = q;
  p.in[1] = k;
  p.out[0] = q_out;
  p.out[1] = k_out;
  p.in_stride[0] = q_stride;
  p.in_stride[1] = k_stride;
  p.out_stride[0] = q_out_stride;
  p.out_stride[1] = k_out_stride;
  p.positions = positions;
  p.turns = rope->turns;
  p.tokens = tokens;
  p.heads = num_heads;
  p.tensors = k ? 2 : 1;
  p.rotary = rope->rotary_dim;
  p.magnitude = rope->magnitude;
  p.sign = backward ? -1.0f : 1.0f;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == HSTU_DTYPE_F16
                            ? hstu::launch_rope_typed<__half>(p, head_dim, rope->interleaved != 0, cs)
                            : hstu::launch_rope_typed<__nv_bfloat16>(p, head_dim, rope->interleaved != 0, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"

// Root-mean-square norms of rows, with the residual's addition in front, a gate
// behind, and an output in 16 or 8 bits; their gradients; and rows quantised as
// they are.
//
//   forward   h = x + residual, rounded to the rows' type, which is how the
//             stream is kept; rstd = (mean(h^2) + eps)^(-1/2); y = h rstd weight gate.
//             The norm is that of the h that is kept, so that the backward, which
//             reads it, differentiates the very function that ran.
//             8-bit output: e4m3 codes of y under a power of two for each row,
//             the cache's rule.
//   backward  with u = h rstd and t = dy gate weight:
//             dx = rstd (t - u mean(t u)) + dh,  dgate = dy u weight,
//             dweight = the sum over rows of dy gate u.
//
// A row lies in the registers of the 8 to 512 threads that share it, so it is
// read and written once, with one reduction (two for 8 bits) by shuffles and,
// above 1024 columns, shared memory. Sums are in 32 bits. The backward's blocks
// take rows in turn and keep their part of dweight in registers; the blocks'
// parts are added in order by a second kernel (no atomics).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache.cuh"
#include "layer.cuh"
#include "pairs.cuh"

namespace hstu {
namespace {

constexpr int kNormMaxWidth = 8192;
constexpr int kNormMaxBlocks = 152 * 4;  // of the backward: parts of dweight
constexpr float kMaxFinite = 3.402823466e38f;

// What a kernel makes of its rows.
constexpr int kNorm16 = 0, kNorm8 = 1, kCodes = 2;

struct NormParams {
  const void* x;
  const void* residual;  // nullable
  const void* gate;      // nullable
  const void* weight;
  void* y;         // 16-bit rows or codes
  uint8_t* scale;  // 8-bit output
  void* h;         // nullable
  float* rstd;     // nullable
  int64_t x_stride, residual_stride, gate_stride, rows;
  int32_t width;
  float eps;
};

// Sum or maximum over the RT threads of a row; every thread of the block calls it.
// `shared` has a value for each warp and is not in use by the reduction before.
template <int RT, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* shared) {
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int off = 1; off < (RT < 32 ? RT : 32); off <<= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, off));
  if (RT <= 32) return v;
  constexpr int kWarps = RT < 32 ? 1 : RT / 32;
  const int warp = threadIdx.x >> 5, first = warp / kWarps * kWarps;
  if ((threadIdx.x & 31) == 0) shared[warp] = v;
  __syncthreads();
  v = shared[first];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = join(v, shared[first + w]);
  return v;
}

template <int RT>
constexpr int norm_threads() { return RT > 128 ? RT : 128; }

// RT threads a row, V chunks of 8 columns a thread.
template <typename T, int RT, int V, int OUT>
__global__ void __launch_bounds__(norm_threads<RT>()) norm_kernel(const NormParams p) {
  chain();
  __shared__ float shared[2][RT > 32 ? norm_threads<RT>() / 32 : 1];
  const int t = threadIdx.x % RT;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (norm_threads<RT>() / RT) + threadIdx.x / RT;
  const bool live = r < p.rows;
  uint4 xv[V], rv[V], gv[V], wv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (t + i * RT) * 8;
    xv[i] = rv[i] = gv[i] = wv[i] = make_uint4(0, 0, 0, 0);
    if (!live || col >= p.width) continue;
    xv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + r * p.x_stride + col);
    if (OUT == kCodes) continue;
    if (p.residual)
      rv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.residual) + r * p.residual_stride + col);
    if (p.gate) gv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.gate) + r * p.gate_stride + col);
    wv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.weight) + col);
  }
  float rstd = 1.0f;
  if (OUT != kCodes) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float f[8];
      unpack8<T>(xv[i], f);
      if (p.residual) {
        float g[8];
        unpack8<T>(rv[i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += g[e];
        xv[i] = pack8<T>(f);
        unpack8<T>(xv[i], f);  // h as it is kept
        const int col = (t + i * RT) * 8;
        if (p.h && live && col < p.width)
          *reinterpret_cast<uint4*>(static_cast<T*>(p.h) + r * p.width + col) = xv[i];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
    }
    sum = row_reduce<RT, false>(sum, shared[0]);
    rstd = 1.0f / sqrtf(sum / static_cast<float>(p.width) + p.eps);
    if (p.rstd && live && t == 0) p.rstd[r] = rstd;
  }
  uint64_t y[V][4];
  float top = 0.0f;  // largest magnitude; NaN is passed over
  const uint64_t rr = pair_of(rstd, rstd);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w}, ww[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w},
                   gw[4] = {gv[i].x, gv[i].y, gv[i].z, gv[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      y[i][e] = unpack_pair<T>(xw[e]);
      if (OUT != kCodes) {
        y[i][e] = pair_mul(y[i][e], pair_mul(rr, unpack_pair<T>(ww[e])));
        if (p.gate) y[i][e] = pair_mul(y[i][e], unpack_pair<T>(gw[e]));
      }
      if (OUT != kNorm16) {
        float a, b;
        pair_split(y[i][e], a, b);
        top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
      }
    }
    const int col = (t + i * RT) * 8;
    if (OUT == kNorm16 && live && col < p.width)
      *reinterpret_cast<uint4*>(static_cast<T*>(p.y) + r * p.width + col) =
          make_uint4(pack_pair<T>(y[i][0]), pack_pair<T>(y[i][1]), pack_pair<T>(y[i][2]), pack_pair<T>(y[i][3]));
  }
  if (OUT == kNorm16) return;
  // The scale goes by the finite values: a row with an infinity looks for its largest again.
  // (Every row of the block does then, for the barriers' sake; nothing changes for the others.)
  top = row_reduce<RT, true>(top, shared[1]);
  const bool infinite = top > kMaxFinite;
  const bool again = RT == norm_threads<RT>() ? infinite  // a row a block
                     : RT > 32                ? __syncthreads_or(infinite)
                                              : __any_sync(0xffffffffu, infinite);
  if (again) {
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a, b;
        pair_split(y[i][e], a, b);
        top = fmaxf(top, fmaxf(fabsf(a) <= kMaxFinite ? fabsf(a) : 0.0f, fabsf(b) <= kMaxFinite ? fabsf(b) : 0.0f));
      }
    top = row_reduce<RT, true>(top, shared[0]);
  }
  const uint32_t byte = scale_byte(top);
  const float inv = __uint_as_float((254u - byte) << 23);  // 2^(127 - byte), exact
  const uint64_t ii = pair_of(inv, inv);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (t + i * RT) * 8;
    if (!live || col >= p.width) continue;
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      pair_split(pair_mul(y[i][e], ii), a, b);
      if (infinite) {  // infinities become NaN, as NaN does
        a = fabsf(a) <= kMaxFinite ? a : __uint_as_float(0x7fc00000u);
        b = fabsf(b) <= kMaxFinite ? b : __uint_as_float(0x7fc00000u);
      }
      c[e] = e4m3x2(a, b);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + r * p.width + col) =
        make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
  if (live && t == 0) p.scale[r] = static_cast<uint8_t>(byte);
}

struct NormBwdParams {
  const void* dy;
  const void* h;
  const float* rstd;
  const void* weight;
  const void* gate;  // nullable
  const void* dh;    // nullable
  void* dx;
  void* dgate;  // nullable
  float* part;  // (blocks, width)
  int64_t dy_stride, h_stride, gate_stride, dh_stride, rows;
  int32_t width;
};

constexpr int kNormBwdThreads = 256;
template <int RT>
constexpr int norm_bwd_threads() { return RT > kNormBwdThreads ? RT : kNormBwdThreads; }

template <typename T, int RT, int V, bool GATE>
__global__ void __launch_bounds__(norm_bwd_threads<RT>()) norm_bwd_kernel(const NormBwdParams p) {
  chain();
  constexpr int kThreads = norm_bwd_threads<RT>(), kGroups = kThreads / RT;
  __shared__ float shared[2][kThreads / 32];  // in turn: one barrier a row
  __shared__ float red[kGroups > 1 ? RT * V * 8 : 1];
  const int t = threadIdx.x % RT, group = threadIdx.x / RT;
  uint4 wv[V];
  float acc[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int col = (t + i * RT) * 8;
    wv[i] = make_uint4(0, 0, 0, 0);
    if (col < p.width) wv[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.weight) + col);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
  }
  const float inv_width = 1.0f / static_cast<float>(p.width);
  // A row's loads are on their way while the row before is worked on (81920 rows of
  // 512: 51 us, without 56 us); with a gate the registers for it cost more blocks than
  // it gains (65 us without, 78 us).
  constexpr bool kAhead = !GATE;
  uint4 dv[V], hv[V], gv[V], ev[V];
  float rstd = 0.0f;
  auto read_row = [&](int64_t r, uint4 (&d)[V], uint4 (&h)[V], uint4 (&g)[V], uint4 (&e)[V], float& s) {
    s = r < p.rows ? p.rstd[r] : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (t + i * RT) * 8;
      d[i] = h[i] = g[i] = e[i] = make_uint4(0, 0, 0, 0);
      if (r >= p.rows || col >= p.width) continue;
      d[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.dy) + r * p.dy_stride + col);
      h[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.h) + r * p.h_stride + col);
      if (GATE) g[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.gate) + r * p.gate_stride + col);
      if (p.dh) e[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.dh) + r * p.dh_stride + col);
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  if (kAhead) read_row(static_cast<int64_t>(blockIdx.x) * kGroups + group, dv, hv, gv, ev, rstd);
  // All groups of a block go around together: the reduction has barriers.
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups; r0 < p.rows; r0 += step, turn ^= 1) {
    const int64_t r = r0 + group;
    const bool live = r < p.rows;
    uint4 next_d[V], next_h[V], next_g[V], next_e[V];
    float next_rstd;
    if (kAhead) read_row(r + step, next_d, next_h, next_g, next_e, next_rstd);
    else read_row(r, dv, hv, gv, ev, rstd);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float d[8], u[8], w[8], g[8];
      unpack8<T>(dv[i], d);
      unpack8<T>(hv[i], u);
      unpack8<T>(wv[i], w);
      if (GATE) unpack8<T>(gv[i], g);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[e] *= rstd;
        const float a = GATE ? d[e] * g[e] : d[e];
        acc[i][e] = fmaf(a, u[e], acc[i][e]);
        sum = fmaf(a * w[e], u[e], sum);
        if (GATE) d[e] *= u[e] * w[e];
      }
      const int col = (t + i * RT) * 8;
      if (GATE && live && col < p.width) store8(static_cast<T*>(p.dgate) + r * p.width + col, d);
    }
    const float mean = row_reduce<RT, false>(sum, shared[turn]) * inv_width;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (t + i * RT) * 8;
      if (!live || col >= p.width) continue;
      float d[8], u[8], w[8], g[8];
      unpack8<T>(dv[i], d);
      unpack8<T>(hv[i], u);
      unpack8<T>(wv[i], w);
      if (GATE) unpack8<T>(gv[i], g);
      float x[8];
      unpack8<T>(ev[i], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = (GATE ? d[e] * g[e] : d[e]) * w[e];
        x[e] += rstd * (a - u[e] * rstd * mean);
      }
      store8(static_cast<T*>(p.dx) + r * p.width + col, x);
    }
    if (!kAhead) continue;
    rstd = next_rstd;
#pragma unroll
    for (int i = 0; i < V; ++i) dv[i] = next_d[i], hv[i] = next_h[i], gv[i] = next_g[i], ev[i] = next_e[i];
  }
  // The groups' sums, in their order.
  if (kGroups > 1) {
    for (int g = 0; g < kGroups; ++g) {
      if (group == g)
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float& s = red[(t + i * RT) * 8 + e];
            s = g == 0 ? acc[i][e] : s + acc[i][e];
          }
      __syncthreads();
    }
  }
  if (group == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int col = (t + i * RT) * 8;
      if (col >= p.width) continue;
      if (kGroups > 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = red[col + e];
      store8(p.part + static_cast<int64_t>(blockIdx.x) * p.width + col, acc[i]);
    }
  }
}

// dweight[col] = the blocks' parts in order: warp w of a block adds parts w, w + 32,
// ... of 32 columns, then the warps' sums are added in order.
template <typename T>
__global__ void __launch_bounds__(1024) norm_fold_kernel(const float* part, int blocks, int width, void* dweight) {
  chain();
  __shared__ float red[32][33];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, col = blockIdx.x * 32 + l;
  float s = 0.0f;
  if (col < width)
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * width + col];
  red[w][l] = s;
  __syncthreads();
  if (w == 0 && col < width) {
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < 32; ++x) sum += red[x][l];
    static_cast<uint16_t*>(dweight)[col] = static_cast<uint16_t>(Elem<T>::pack2(sum, 0.0f) & 0xffffu);
  }
}

// Threads of a row and chunks a thread. Forward: the fewest threads whose registers
// hold the row, so that reductions stay inside a warp up to 1024 columns and take few
// warps above (16381 rows of 2048 with a residual into 8 bits: 36 us, 42 us with a chunk
// a thread); 8 and 16 threads for narrow rows (heads of 64 and 128, of a contiguous (T, H, D)
// tensor seen as T H rows), where a whole warp would leave most of its lanes without
// columns.
// The backward holds up to four rows and its part of dweight besides: one or two
// chunks a thread, so that several blocks fit an SM (32749 rows of 1024, with a gate:
// 72 us with four chunks a lane and one block an SM, 65 us with a chunk a thread, 62 us with
// two; 16381 rows of 2048 with dh 46 us so, 51 us with a chunk a thread).
template <bool BACKWARD, typename F>
cudaError_t by_width(int width, F&& f) {
  using std::integral_constant;
  auto call = [&](auto rt, auto v) { return f(rt, v); };
  if (width <= 64) return call(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (width <= 128) return call(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (width <= 256) return call(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (width <= 512) return call(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  if constexpr (BACKWARD) {
    if (width <= 1024) return call(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (width <= 2048) return call(integral_constant<int, 128>{}, integral_constant<int, 2>{});
    if (width <= 4096) return call(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    return call(integral_constant<int, 512>{}, integral_constant<int, 2>{});
  } else {
    if (width <= 1024) return call(integral_constant<int, 32>{}, integral_constant<int, 4>{});
    if (width <= 2048) return call(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    if (width <= 4096) return call(integral_constant<int, 128>{}, integral_constant<int, 4>{});
    return call(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  }
}

template <typename T, int OUT>
cudaError_t launch_norm(const NormParams& p, cudaStream_t stream) {
  return by_width<false>(p.width, [&](auto rt, auto v) {
    constexpr int RT = decltype(rt)::value, V = decltype(v)::value;
    constexpr int per = norm_threads<RT>() / RT;
    return launch_chained(norm_kernel<T, RT, V, OUT>, dim3(static_cast<unsigned>((p.rows + per - 1) / per)),
                          norm_threads<RT>(), 0, stream, p);
  });
}
template <int OUT>
cudaError_t launch_norm_typed(const NormParams& p, int dtype, cudaStream_t stream) {
  return dtype == HSTU_DTYPE_F16 ? launch_norm<__half, OUT>(p, stream) : launch_norm<__nv_bfloat16, OUT>(p, stream);
}

template <typename T>
cudaError_t launch_norm_bwd(const NormBwdParams& p, void* dweight, cudaStream_t stream) {
  int blocks = 0;
  cudaError_t e = by_width<true>(p.width, [&](auto rt, auto v) {
    constexpr int RT = decltype(rt)::value, V = decltype(v)::value;
    constexpr int threads = norm_bwd_threads<RT>(), per = threads / RT;
    auto kernel = p.gate ? norm_bwd_kernel<T, RT, V, true> : norm_bwd_kernel<T, RT, V, false>;
    // as many blocks as run at a time
    static std::atomic<int> resident[2];
    int fit = resident[p.gate != nullptr].load();
    if (fit == 0) {
      const cudaError_t q = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, threads, 0);
      if (q != cudaSuccess) return q;
      fit = std::max(1, std::min(fit, kNormMaxBlocks / 152));
      resident[p.gate != nullptr].store(fit);
    }
    blocks = static_cast<int>(std::min<int64_t>((p.rows + per - 1) / per, 152 * fit));
    return launch_chained(kernel, dim3(blocks), threads, 0, stream, p);
  });
  if (e != cudaSuccess) return e;
  return launch_chained(norm_fold_kernel<T>, dim3((p.width + 31) / 32), 1024, 0, stream,
                        static_cast<const float*>(p.part), blocks, p.width, dweight);
}

hstu_status_t norm_checks(int64_t rows, int width) {
  if (rows < 0 || rows > INT32_MAX || width < 1) return HSTU_ERR_INVALID_ARG;
  return width % 8 != 0 || width > kNormMaxWidth ? HSTU_ERR_UNSUPPORTED : HSTU_OK;
}

}  // namespace
}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_attn_rms_norm(const void* x, int64_t x_stride, const void* residual,
                                          int64_t residual_stride, const void* gate, int64_t gate_stride,
                                          const void* weight, int64_t rows, int32_t width, int32_t dtype, float eps,
                                          void* y, uint8_t* y_scale, void* h, float* rstd, void* stream) {
  using namespace hstu;
  const hstu_status_t st = norm_checks(rows, width);
  if (st != HSTU_OK) return st;
  if (!row_dtype_ok(dtype)) return HSTU_ERR_UNSUPPORTED;
  if (!(eps >= 0.0f) || eps > kMaxFinite) return HSTU_ERR_INVALID_ARG;
  if (rows == 0) return HSTU_OK;
  if (!rows_ok(x, x_stride, 1, width) || (residual && !rows_ok(residual, residual_stride, 1, width)) ||
      (gate && !rows_ok(gate, gate_stride, 1, width)) || !aligned_to(weight, 16) || !aligned_to(y, 16) ||
      (residual == nullptr) != (h == nullptr) || (h && !aligned_to(h, 16)) || (rstd && !aligned_to(rstd, 4)))
    return HSTU_ERR_INVALID_ARG;
  const int64_t w = int64_t{width} * 2, yw = y_scale ? width : w;
  // h may be the residual's or x's own rows: a row's threads have read all of it before they write.
  const bool over_r = h && h == residual && residual_stride == width, over_x = h && h == x && x_stride == width;
  const RowSpan in[] = {{over_x ? nullptr : x, 2 * x_stride, w, rows},
                        {over_r ? nullptr : residual, 2 * residual_stride, w, rows},
                        {gate, 2 * gate_stride, w, rows},
                        {weight, w, w, 1}},
                out[] = {{y, yw, yw, rows}, {y_scale, 1, 1, rows}, {h, w, w, rows}, {rstd, 4, 4, rows}};
  if (outputs_meet(in, out)) return HSTU_ERR_INVALID_ARG;
  NormParams p{};
  p.x = x;
  p.residual = residual;
  p.gate = gate;
  p.weight = weight;
  p.y = y;
  p.scale = y_scale;
  p.h = h;
  p.rstd = rstd;
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.gate_stride = gate_stride;
  p.rows = rows;
  p.width = width;
  p.eps = eps;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = y_scale ? launch_norm_typed<kNorm8>(p, dtype, cs) : launch_norm_typed<kNorm16>(p, dtype, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API hstu_status_t hstu_attn_quantise_rows(const void* x, int64_t x_stride, int64_t rows, int32_t width,
                                               int32_t dtype, uint8_t* codes, uint8_t* scale, void* stream) {
  using namespace hstu;
  const hstu_status_t st = norm_checks(rows, width);
  if (st != HSTU_OK) return st;
  if (!row_dtype_ok(dtype)) return HSTU_ERR_UNSUPPORTED;
  if (rows == 0) return HSTU_OK;
  if (!rows_ok(x, x_stride, 1, width) || !aligned_to(codes, 16) || !scale) return HSTU_ERR_INVALID_ARG;
  const RowSpan in[] = {{x, 2 * x_stride, int64_t{width} * 2, rows}},
                out[] = {{codes, width, width, rows}, {scale, 1, 1, rows}};
  if (outputs_meet(in, out)) return HSTU_ERR_INVALID_ARG;
  NormParams p{};
  p.x = x;
  p.x_stride = x_stride;
  p.y = codes;
  p.scale = scale;
  p.rows = rows;
  p.width = width;
  return launch_norm_typed<kCodes>(p, dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HSTU_OK
                                                                                              : HSTU_ERR_CUDA;
}

HSTU_API size_t hstu_attn_rms_norm_workspace_size(int64_t rows, int32_t width) {
  if (hstu::norm_checks(rows, width) != HSTU_OK) return 0;
  const int64_t blocks = rows < hstu::kNormMaxBlocks ? (rows < 1 ? 1 : rows) : hstu::kNormMaxBlocks;
  return hstu::align_up(static_cast<size_t>(blocks) * width * 4, 256);
}

HSTU_API hstu_status_t hstu_attn_rms_norm_bwd(const void* dy, int64_t dy_stride, const void* h, int64_t h_stride,
                                              const float* rstd, const void* weight, const void* gate,
                                              int64_t gate_stride, const void* dh, int64_t dh_stride, int64_t rows,
                                              int32_t width, int32_t dtype, void* dx, void* dweight, void* dgate,
                                              void* ws, size_t ws_bytes, void* stream) {
  using namespace hstu;
  const hstu_status_t st = norm_checks(rows, width);
  if (st != HSTU_OK) return st;
  if (!row_dtype_ok(dtype)) return HSTU_ERR_UNSUPPORTED;
  if (!aligned_to(dweight, 16)) return HSTU_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t w = int64_t{width} * 2;
  if (rows > 0) {
    if (!rows_ok(dy, dy_stride, 1, width) || !rows_ok(h, h_stride, 1, width) || !aligned_to(rstd, 4) ||
        !aligned_to(weight, 16) || (gate && !rows_ok(gate, gate_stride, 1, width)) ||
        (dh && !rows_ok(dh, dh_stride, 1, width)) || !aligned_to(dx, 16) || (gate == nullptr) != (dgate == nullptr) ||
        (dgate && !aligned_to(dgate, 16)))
      return HSTU_ERR_INVALID_ARG;
    const RowSpan in[] = {{dy, 2 * dy_stride, w, rows}, {h, 2 * h_stride, w, rows},       {rstd, 4, 4, rows},
                          {weight, w, w, 1},            {gate, 2 * gate_stride, w, rows}, {dh, 2 * dh_stride, w, rows}},
                  out[] = {{dx, w, w, rows}, {dweight, w, w, 1}, {dgate, w, w, rows}};
    if (outputs_meet(in, out)) return HSTU_ERR_INVALID_ARG;
  }
  if (!aligned_to(ws, 256) || ws_bytes < hstu_attn_rms_norm_workspace_size(rows, width)) return HSTU_ERR_WORKSPACE;
  if (rows == 0)  // no rows: dweight is zero
    return cudaMemsetAsync(dweight, 0, static_cast<size_t>(w), cs) == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
  NormBwdParams p{};
  p.dy = dy;
  p.h = h;
  p.rstd = rstd;
  p.weight = weight;
  p.gate = gate;
  p.dh = dh;
  p.dx = dx;
  p.dgate = dgate;
  p.part = static_cast<float*>(ws);
  p.dy_stride = dy_stride;
  p.h_stride = h_stride;
  p.gate_stride = gate_stride;
  p.dh_stride = dh_stride;
  p.rows = rows;
  p.width = width;
  const cudaError_t e =
      dtype == HSTU_DTYPE_F16 ? launch_norm_bwd<__half>(p, dweight, cs) : launch_norm_bwd<__nv_bfloat16>(p, dweight, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"

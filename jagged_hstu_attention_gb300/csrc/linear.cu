// Linear maps of rows with a fused epilogue, and their gradients.
//
//   forward   z = x w^T + bias, y = act(z) + residual: one tcgen05 product
//             whose epilogue holds everything else, 16-bit or 8-bit operands;
//   backward  g = dy act'(z) and the column sums of g (one elementwise kernel, parts
//             of row chunks added in order), then dx = g w and dw = g^T x on
//             tcgen05, whose operands have 16 bits: g is rounded to them, half a
//             step of relative error in each term of their sums. (The column sums, the bias
//             gradient, are of g in 32 bits.) Without an
//             activation g is dy itself, read in place. dw, whose K is the number
//             of rows, splits K over the SMs; its fp32 parts are added in order.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "layer.cuh"
#include "linear.cuh"

namespace hstu {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradChunks = 152 * 4;
constexpr int kGradRows = 4;  // of a thread, on their way at once
constexpr int kPairs = 76;

// The blocks of the activation's gradient: rows in chunks of at least kGradRows a thread,
// all columns a block where those are blocks enough, else columns evenly in parts of 512, and
// chunks of fewer rows until there is a block for each SM. (33047 rows of 3584 columns
// take 109 us in whole rows and 115 us in parts, 61 rows of 2584 columns 23 us and 3.9. Half as many
// chunks of 3584 columns, all on their way at once, took the backward 240 us, not 202.) A chunk's
// column sums are one part of the bias gradient.
struct GradGrid {
  int col_blocks, groups, rows_at_once, chunks;
};
inline GradGrid grad_grid(int64_t rows, int cols) {
  auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  GradGrid g;
  for (int widest = kGradThreads; widest >= kGradThreads / 4; widest /= 4) {
    g.col_blocks = static_cast<int>(up(cols / 8, widest));
    g.groups = static_cast<int>(up(cols / 8, g.col_blocks));
    g.rows_at_once = kGradThreads / g.groups;
    const int64_t few = std::max(152 / g.col_blocks, 1);
    const int64_t full = up(rows, kGradRows * g.rows_at_once), thin = std::min(up(rows, g.rows_at_once), few);
    g.chunks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kGradChunks, std::max(full, thin))));
    if (full * g.col_blocks >= kGradChunks) break;
  }
  return g;
}

// dy act'(z) of a pair: with p = 1 / (1 + exp(-u)), act' = p (1 + z (1 - p) u').
template <int ACT>
__device__ __forceinline__ uint64_t act_grad2(uint64_t z, uint64_t dy) {
  if (ACT == HSTU_ACT_NONE) return dy;
  if (ACT == HSTU_ACT_RELU) {
    float a, b, c, d;
    pair_split(z, a, b);
    pair_split(dy, c, d);
    return pair_of(a > 0.0f ? c : 0.0f, b > 0.0f ? d : 0.0f);
  }
  // (Past 64, where p is 1, z counts as 64: its square stays finite.)
  float a, b;
  pair_split(z, a, b);
  asm("min.NaN.f32 %0, %0, 0f42800000;" : "+f"(a));
  asm("min.NaN.f32 %0, %0, 0f42800000;" : "+f"(b));
  z = pair_of(max_nan(a, kLowest<ACT>), max_nan(b, kLowest<ACT>));
  uint64_t e;
  const uint64_t p = sigmoid_of<ACT>(z, e);
  uint64_t slope = pair_mul(z, pair_mul(e, p));  // 1 - p = p exp(-u), which nothing cancels in
  if (ACT == HSTU_ACT_GELU)
    slope = pair_mul(slope, pair_fma(pair_mul(z, z), pair_of(3.0f * kGeluA * kGeluB, 3.0f * kGeluA * kGeluB),
                                     pair_of(kGeluA, kGeluA)));
  return pair_mul(dy, pair_mul(p, pair_add(slope, pair_of(1.0f, 1.0f))));
}

struct GradParams {
  const void* dy;
  const void* z;  // without an activation not read: g = dy, nothing is written but the sums
  void* g;
  float* part;  // (chunks, cols)
  int32_t* header;
  int64_t dy_stride, rows;
  int32_t cols;
  int32_t groups, rows_at_once;
};

// A block takes a chunk of rows of its columns, 8 columns a thread, kGradRows rows on their way.
template <typename T, int ACT>
__global__ void __launch_bounds__(kGradThreads, 4) linear_grad_kernel(const GradParams p) {
  chain();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.header[kHdrErr] = 0;  // the products behind may set it
  __shared__ float red[8][kGradThreads];
  const int gy = p.groups, rpi = p.rows_at_once;
  const int lane_row = threadIdx.x / gy, col = (blockIdx.y * gy + threadIdx.x % gy) * 8;
  const bool active = lane_row < rpi && col < p.cols;
  const int64_t step = int64_t{rpi} * gridDim.x, per = (p.rows + step - 1) / step * rpi;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * per, r1 = min(r0 + per, p.rows);
  uint64_t sums[4] = {};
  auto one = [&](uint4 zv, uint4 dv, int64_t to) {
    // the sums are those of g in 32 bits; only the products' operand is rounded
    auto two = [&](int e, uint32_t zw, uint32_t dw) {
      const uint64_t g = act_grad2<ACT>(unpack_pair<T>(zw), unpack_pair<T>(dw));
      sums[e] = pair_add(sums[e], g);
      return pack_pair<T>(g);
    };
    dv.x = two(0, zv.x, dv.x);
    dv.y = two(1, zv.y, dv.y);
    dv.z = two(2, zv.z, dv.z);
    dv.w = two(3, zv.w, dv.w);
    if (ACT != HSTU_ACT_NONE) *reinterpret_cast<uint4*>(static_cast<T*>(p.g) + to) = dv;
  };
  if (active && r0 + lane_row < r1) {
    // Of the thread's next row; its rows are rpi apart.
    int64_t at = (r0 + lane_row) * p.cols + col, dy_at = (r0 + lane_row) * p.dy_stride + col;
    const int64_t at_step = int64_t{rpi} * p.cols, dy_step = rpi * p.dy_stride;
    int left = static_cast<int>((r1 - r0 - lane_row + rpi - 1) / rpi);
    auto some = [&](auto all) {  // kGradRows rows, or those there are
      uint4 zv[kGradRows], dv[kGradRows];
#pragma unroll
      for (int k = 0; k < kGradRows; ++k) {
        if (!all && k >= left) break;
        zv[k] = make_uint4(0, 0, 0, 0);
        if (ACT != HSTU_ACT_NONE) zv[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.z) + at + k * at_step);
        dv[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.dy) + dy_at + k * dy_step);
      }
#pragma unroll
      for (int k = 0; k < kGradRows; ++k)
        if (all || k < left) one(zv[k], dv[k], at + k * at_step);
    };
    for (; left >= kGradRows; left -= kGradRows) {
      some(std::true_type{});
      at += kGradRows * at_step;
      dy_at += kGradRows * dy_step;
    }
    if (left > 0) some(std::false_type{});
  }
  float sum[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) pair_split(sums[e], sum[2 * e], sum[2 * e + 1]);
#pragma unroll
  for (int e = 0; e < 8; ++e) red[e][threadIdx.x] = sum[e];
  __syncthreads();
  // Rows of threads meet in halves (32163 rows of 16 columns have 128 of them).
  for (int s = 1 << (31 - __clz(max(rpi - 1, 1))); s > 0; s >>= 1) {
    if (lane_row < s && lane_row + s < rpi)
#pragma unroll
      for (int e = 0; e < 8; ++e) red[e][threadIdx.x] = sum[e] += red[e][threadIdx.x + s * gy];
    __syncthreads();
  }
  if (active && lane_row == 0) store8(p.part + static_cast<int64_t>(blockIdx.x) * p.cols + col, sum);
}

// Ends the backward: dw from the fp32 parts of K's splits, 8 elements a thread (blocks
// [0, dw_blocks)), where there are many splits `slices` threads that take a part of them
// each; dbias from the chunks' parts in order, 32 columns a block, a part in 32 a warp (the
// blocks behind).
constexpr int kFoldThreads = 1024, kFoldSplits = 8;  // of a slice, about
struct FoldParams {
  const float* dw_part;
  void* dw;
  const float* bias_part;
  void* dbias;
  int64_t elems;  // of dw
  int32_t splits, slices, chunks, cols, dw_blocks;
};
template <typename T>
__global__ void __launch_bounds__(kFoldThreads) linear_fold_kernel(const FoldParams p) {
  chain();
  if (static_cast<int>(blockIdx.x) < p.dw_blocks) {
    __shared__ float4 slice[kFoldThreads][2];
    const int width = kFoldThreads / p.slices, q = threadIdx.x / width;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * width + threadIdx.x % width) * 8;
    float acc[8] = {};
    if (i < p.elems) {
      const int s1 = p.splits * (q + 1) / p.slices;
#pragma unroll 4
      for (int s = p.splits * q / p.slices; s < s1; ++s) {
        float f[8];
        load8(p.dw_part + s * p.elems + i, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[e];
      }
    }
    if (p.slices > 1) {
      slice[threadIdx.x][0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      slice[threadIdx.x][1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      __syncthreads();
      if (q > 0) return;
      for (int x = 1; x < p.slices; ++x) {
        const float4 lo = slice[x * width + threadIdx.x][0], hi = slice[x * width + threadIdx.x][1];
        acc[0] += lo.x, acc[1] += lo.y, acc[2] += lo.z, acc[3] += lo.w;
        acc[4] += hi.x, acc[5] += hi.y, acc[6] += hi.z, acc[7] += hi.w;
      }
    }
    if (i < p.elems) store8(static_cast<T*>(p.dw) + i, acc);
    return;
  }
  __shared__ float red[32][33];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, col = (blockIdx.x - p.dw_blocks) * 32 + l;
  float s = 0.0f;
  if (col < p.cols)
#pragma unroll 8
    for (int c = w; c < p.chunks; c += 32) s += p.bias_part[static_cast<int64_t>(c) * p.cols + col];
  red[w][l] = s;
  __syncthreads();
  if (w == 0 && col < p.cols) {
    float sum = 0.0f;
#pragma unroll
    for (int x = 0; x < 32; ++x) sum += red[x][l];
    static_cast<uint16_t*>(p.dbias)[col] = static_cast<uint16_t>(Elem<T>::pack2(sum, 0.0f) & 0xffffu);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Boxes of 128 bytes x box_rows of a row-major (rows, cols) operand; what lies outside it
// reads as zeros.
constexpr int kDtypeCodes = -1;  // 8-bit
bool box_map(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int64_t stride, int dtype, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool codes = dtype == kDtypeCodes;
  const CUtensorMapDataType type = codes                      ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == HSTU_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * (codes ? 1 : 2)};
  cuuint32_t box[2] = {codes ? 128u : 64u, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

hstu_status_t linear_checks(int64_t rows, int d_in, int d_out, int act, bool codes) {
  if (rows < 0 || rows > INT32_MAX - 1024 || d_in < 1 || d_out < 1) return HSTU_ERR_INVALID_ARG;
  if (d_in % (codes ? 16 : 8) || d_out % 8 || d_in > 65536 || d_out > 65536) return HSTU_ERR_UNSUPPORTED;
  if (act < HSTU_ACT_NONE || act > HSTU_ACT_RELU) return HSTU_ERR_UNSUPPORTED;
  // tiles are numbered in 32 bits
  const int64_t most = d_in > d_out ? d_in : d_out;
  if ((rows / kTileM + 1) * (most / kTileN + 1) > INT32_MAX / 2) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

// A model of the time of a product on pairs of SMs, in units of 10 ns. Tiles of half the
// columns take three quarters of a whole one's time, and so pay while there are pairs
// left for twice as many (512 x 4096 x 4096: 19.0 and 25.6 us; 2000 rows 63 and 44).
int64_t pairs_cost(int64_t rows, int outputs, int64_t k_bytes, bool narrow) {
  const int tn = narrow ? kTileN / 2 : kTileN;
  const int64_t tiles = (rows + kTileM - 1) / kTileM * ((outputs + tn - 1) / tn), nk = (k_bytes + 127) / 128;
  return 330 + (tiles + kPairs - 1) / kPairs * (narrow ? 110 + 23 * nk : 150 + 31 * nk);
}
bool narrow_tiles(int64_t rows, int outputs, int64_t k_bytes) {
  return pairs_cost(rows, outputs, k_bytes, true) < pairs_cost(rows, outputs, k_bytes, false);
}
// Whether a product goes to the kernel for few rows: where its model of the time is below
// that of pairs of SMs (512 x 2048: 64 rows take 5.1 us there and 6.4 us on pairs, 512 rows 9.8
// and 7.6; 4096 x 4096: 64 rows 11.8 and 23 us, 384 rows 49 and 24), and its tiles run
// at the same time, or there are no more rows than one tile may have.
bool few_rows(int64_t rows, int outputs, int64_t k_bytes) {
  const FewPlan plan = few_plan(rows, outputs, k_bytes);
  return plan.cost <= std::min(pairs_cost(rows, outputs, k_bytes, false), pairs_cost(rows, outputs, k_bytes, true)) &&
         (rows <= kFewRows || few_tiles(rows, outputs, plan.rows_tile) <= 152);
}

// Splits of dw's K: those that take the least time, in 64-row blocks: the tiles of the
// busiest pair, each split's fp32 tile counting as four blocks, and the sums' way through
// the fold, at some 400000 values a block. (46120 rows of 152 and 200 columns: 45 us for the
// backward with 16 splits, 37 with 73; 81920 of 512 and 2048: 410 with 14, 399 with 9.)
int64_t dw_tiles(int d_in, int d_out) {
  return int64_t{(d_out + kTileM - 1) / kTileM} * ((d_in + kTileN - 1) / kTileN);
}
// Two turns of the pairs at the most.
int most_splits(int64_t rows, int d_in, int d_out) {
  const int64_t fit = std::min<int64_t>(kPairs, std::max<int64_t>(1, 2 * kPairs / dw_tiles(d_in, d_out)));
  return static_cast<int>(std::max<int64_t>(1, std::min(fit, (rows + 63) / 64)));
}
int dw_splits(int64_t rows, int d_in, int d_out) {
  const int64_t tiles = dw_tiles(d_in, d_out), nk = (rows + 63) / 64, elems = int64_t{d_in} * d_out;
  const int most = most_splits(rows, d_in, d_out);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= most; ++s) {
    const int64_t per = (nk + s - 1) / s;
    if ((s - 1) * per >= nk) continue;  // a split without rows
    const int64_t cost = (tiles * s + kPairs - 1) / kPairs * (per + (s > 1 ? 4 : 0)) + (s > 1 ? 8 + s * elems / 400000 : 0);
    if (cost < least) least = cost, best = s;
  }
  return best;
}

// Workspace of the backward: a 256-byte header (error word), g, the bias gradient's
// parts, dw's parts, as many as fewer rows may have.
struct LinearLayout {
  size_t g = 0, part = 0, dw = 0, total = 0;
};
LinearLayout linear_layout(int64_t rows, int d_in, int d_out, int act) {
  LinearLayout l;
  l.g = kHdrWords * 4;
  l.part = l.g + (act != HSTU_ACT_NONE ? align_up(static_cast<size_t>(rows) * d_out * 2, 256) : 0);
  l.dw = l.part + align_up(static_cast<size_t>(grad_grid(rows, d_out).chunks) * d_out * 4, 256);
  const int splits = most_splits(rows, d_in, d_out);
  l.total = l.dw + (splits > 1 ? align_up(static_cast<size_t>(splits) * d_out * d_in * 4, 256) : 0);
  return l;
}

template <typename T>
cudaError_t launch_grad(GradParams p, int act, cudaStream_t stream) {
  const GradGrid g = grad_grid(p.rows, p.cols);
  p.groups = g.groups;
  p.rows_at_once = g.rows_at_once;
  const dim3 grid(g.chunks, g.col_blocks);
  auto kernel = act == HSTU_ACT_SILU   ? linear_grad_kernel<T, HSTU_ACT_SILU>
                : act == HSTU_ACT_GELU ? linear_grad_kernel<T, HSTU_ACT_GELU>
                : act == HSTU_ACT_RELU ? linear_grad_kernel<T, HSTU_ACT_RELU>
                                       : linear_grad_kernel<T, HSTU_ACT_NONE>;
  return launch_chained(kernel, grid, kGradThreads, 0, stream, p);
}

}  // namespace
}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_attn_linear(const void* x, int64_t x_stride, const uint8_t* x_scale, const void* w,
                                        const uint8_t* w_scale, const void* bias, const void* residual,
                                        int64_t residual_stride, int64_t rows, int32_t d_in, int32_t d_out,
                                        int32_t dtype, int32_t act, void* y, void* z, void* ws, size_t ws_bytes,
                                        void* stream) {
  using namespace hstu;
  const bool codes = w_scale != nullptr;
  const hstu_status_t st = linear_checks(rows, d_in, d_out, act, codes);
  if (st != HSTU_OK) return st;
  if (!row_dtype_ok(dtype)) return HSTU_ERR_UNSUPPORTED;
  if (ws && (!aligned_to(ws, 256) || ws_bytes < kHdrWords * 4)) return HSTU_ERR_WORKSPACE;
  const int xe = codes ? 1 : 2;
  if (rows > 0) {
    if (!aligned_to(x, 16) || x_stride < d_in || x_stride * xe % 16 != 0 || !aligned_to(w, 16) ||
        (x_scale != nullptr) != codes || (codes && !aligned_to(w_scale, 16)) || (bias && !aligned_to(bias, 16)) ||
        (residual && !rows_ok(residual, residual_stride, 1, d_out)) || !aligned_to(y, 16) || (z && !aligned_to(z, 16)))
      return HSTU_ERR_INVALID_ARG;
    const int64_t yw = int64_t{d_out} * 2;
    const RowSpan in[] = {{x, x_stride * xe, int64_t{d_in} * xe, rows},
                          {w, int64_t{d_in} * xe * d_out, int64_t{d_in} * xe * d_out, 1},
                          {x_scale, rows, rows, 1},
                          {w_scale, d_out, d_out, 1},
                          {bias, yw, yw, 1},
                          {residual, 2 * residual_stride, yw, rows}},
                  out[] = {{y, yw, yw, rows}, {z, yw, yw, rows}};
    if (outputs_meet(in, out)) return HSTU_ERR_INVALID_ARG;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (ws && cudaMemsetAsync(ws, 0, kHdrWords * 4, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  if (rows == 0) return HSTU_OK;
  if (few_rows(rows, d_out, int64_t{d_in} * xe)) {
    FewParams p{};
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.residual = residual;
    p.x_scale = x_scale;
    p.w_scale = w_scale;
    p.y = y;
    p.z = z;
    p.header = static_cast<int32_t*>(ws);
    p.x_stride = x_stride * xe;
    p.residual_stride = residual_stride;
    p.k_bytes = int64_t{d_in} * xe;
    p.give_up = handoff_limit() <= 1;
    p.M = static_cast<int32_t>(rows);
    p.N = d_out;
    p.act = act;
    const cudaError_t e = dtype == HSTU_DTYPE_F16 ? launch_few_f16(p, codes, cs) : launch_few_bf16(p, codes, cs);
    return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
  }
  LinearParams p{};
  p.narrow = narrow_tiles(rows, d_out, int64_t{d_in} * xe);
  const int type = codes ? kDtypeCodes : dtype;
  if (!box_map(&p.tm_a, x, rows, d_in, x_stride, type, 128) || !box_map(&p.tm_b, w, d_out, d_in, d_in, type, p.narrow ? 64 : 128))
    return HSTU_ERR_CUDA;
  p.y = y;
  p.z = z;
  p.residual = residual;
  p.residual_stride = residual_stride;
  p.bias = bias;
  p.a_scale = x_scale;
  p.b_scale = w_scale;
  p.header = static_cast<int32_t*>(ws);
  p.handoff_limit_ns = handoff_limit();
  p.M = static_cast<int32_t>(rows);
  p.N = d_out;
  p.K = d_in;
  p.k_splits = 1;
  p.act = act;
  const cudaError_t e =
      dtype == HSTU_DTYPE_F16 ? launch_linear_f16(p, codes, cs) : launch_linear_bf16(p, codes, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API size_t hstu_attn_linear_workspace_size(int64_t rows, int32_t d_in, int32_t d_out, int32_t act) {
  if (hstu::linear_checks(rows, d_in, d_out, act, false) != HSTU_OK) return 0;
  return hstu::linear_layout(rows, d_in, d_out, act).total;
}

HSTU_API hstu_status_t hstu_attn_linear_bwd(const void* dy, int64_t dy_stride, const void* z, const void* x,
                                            int64_t x_stride, const void* w, int64_t rows, int32_t d_in, int32_t d_out,
                                            int32_t dtype, int32_t act, void* dx, void* dw, void* dbias, void* ws,
                                            size_t ws_bytes, void* stream) {
  using namespace hstu;
  const hstu_status_t st = linear_checks(rows, d_in, d_out, act, false);
  if (st != HSTU_OK) return st;
  if (!row_dtype_ok(dtype)) return HSTU_ERR_UNSUPPORTED;
  const bool f16 = dtype == HSTU_DTYPE_F16;
  if (!aligned_to(dw, 16) || (dbias && !aligned_to(dbias, 16))) return HSTU_ERR_INVALID_ARG;
  const int64_t in_w = int64_t{d_in} * 2, out_w = int64_t{d_out} * 2;
  if (rows > 0) {
    if (!rows_ok(dy, dy_stride, 1, d_out) || !rows_ok(x, x_stride, 1, d_in) || !aligned_to(w, 16) ||
        (act != HSTU_ACT_NONE && !aligned_to(z, 16)) || !aligned_to(dx, 16))
      return HSTU_ERR_INVALID_ARG;
    const RowSpan in[] = {{dy, 2 * dy_stride, out_w, rows},
                          {act != HSTU_ACT_NONE ? z : nullptr, out_w, out_w, rows},
                          {x, 2 * x_stride, in_w, rows},
                          {w, in_w * d_out, in_w * d_out, 1}},
                  out[] = {{dx, in_w, in_w, rows}, {dw, in_w * d_out, in_w * d_out, 1}, {dbias, out_w, out_w, 1}};
    if (outputs_meet(in, out)) return HSTU_ERR_INVALID_ARG;
  }
  const LinearLayout l = linear_layout(rows, d_in, d_out, act);
  if (!aligned_to(ws, 256) || ws_bytes < l.total) return HSTU_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const bool grads = act != HSTU_ACT_NONE || dbias;  // the kernel that makes g or its sums clears the error word
  if ((rows == 0 || !grads) && cudaMemsetAsync(base, 0, kHdrWords * 4, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  if (rows == 0) {  // no rows: dw and dbias are zero
    if (cudaMemsetAsync(dw, 0, static_cast<size_t>(in_w) * d_out, cs) != cudaSuccess ||
        (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(out_w), cs) != cudaSuccess))
      return HSTU_ERR_CUDA;
    return HSTU_OK;
  }
  const void* g = dy;
  int64_t g_stride = dy_stride;
  if (grads) {
    GradParams gp{};
    gp.header = reinterpret_cast<int32_t*>(base);
    gp.dy = dy;
    gp.z = act != HSTU_ACT_NONE ? z : nullptr;
    gp.g = base + l.g;
    gp.part = reinterpret_cast<float*>(base + l.part);
    gp.dy_stride = dy_stride;
    gp.rows = rows;
    gp.cols = d_out;
    if ((f16 ? launch_grad<__half>(gp, act, cs) : launch_grad<__nv_bfloat16>(gp, act, cs)) != cudaSuccess)
      return HSTU_ERR_CUDA;
    if (gp.z) {
      g = gp.g;
      g_stride = d_out;
    }
  }
  LinearParams p{};
  p.header = reinterpret_cast<int32_t*>(base);
  p.handoff_limit_ns = handoff_limit();
  p.k_splits = 1;
  // dx (rows x d_in) = g (K = d_out along its rows) w (K down its columns)
  if (few_rows(rows, d_in, int64_t{d_out} * 2)) {
    FewParams fp{};
    fp.x = g;
    fp.w = w;
    fp.y = dx;
    fp.header = p.header;
    fp.x_stride = g_stride * 2;
    fp.k_bytes = int64_t{d_out} * 2;
    fp.give_up = handoff_limit() <= 1;
    fp.M = static_cast<int32_t>(rows);
    fp.N = d_in;
    fp.act = HSTU_ACT_NONE;
    if ((f16 ? launch_few_dx_f16(fp, cs) : launch_few_dx_bf16(fp, cs)) != cudaSuccess) return HSTU_ERR_CUDA;
  } else {
    if (!box_map(&p.tm_a, g, rows, d_out, g_stride, dtype, 128) || !box_map(&p.tm_b, w, d_out, d_in, d_in, dtype, 64))
      return HSTU_ERR_CUDA;
    p.narrow = narrow_tiles(rows, d_in, int64_t{d_out} * 2);
    p.y = dx;
    p.M = static_cast<int32_t>(rows);
    p.N = d_in;
    p.K = d_out;
    if ((f16 ? launch_linear_dx_f16(p, cs) : launch_linear_dx_bf16(p, cs)) != cudaSuccess) return HSTU_ERR_CUDA;
  }
  // dw (d_out x d_in) = g^T x: K = rows, down the columns of both
  if (!box_map(&p.tm_a, g, rows, d_out, g_stride, dtype, 64) || !box_map(&p.tm_b, x, rows, d_in, x_stride, dtype, 64))
    return HSTU_ERR_CUDA;
  p.y = dw;
  p.M = d_out;
  p.N = d_in;
  p.K = static_cast<int32_t>(rows);
  p.k_splits = dw_splits(rows, d_in, d_out);
  p.part = reinterpret_cast<float*>(base + l.dw);
  if ((f16 ? launch_linear_dw_f16(p, cs) : launch_linear_dw_bf16(p, cs)) != cudaSuccess) return HSTU_ERR_CUDA;
  if (p.k_splits == 1 && !dbias) return HSTU_OK;
  FoldParams fp{};
  fp.dw_part = p.part;
  fp.dw = dw;
  fp.bias_part = reinterpret_cast<const float*>(base + l.part);
  fp.dbias = dbias;
  fp.elems = int64_t{d_out} * d_in;
  fp.splits = p.k_splits;
  fp.chunks = grad_grid(rows, d_out).chunks;
  fp.cols = d_out;
  fp.slices = 1;
  while (fp.slices * kFoldSplits < fp.splits) fp.slices *= 2;
  const int64_t width = kFoldThreads / fp.slices;
  fp.dw_blocks = p.k_splits > 1 ? static_cast<int32_t>((fp.elems / 8 + width - 1) / width) : 0;
  const dim3 grid(static_cast<unsigned>(fp.dw_blocks + (dbias ? (d_out + 31) / 32 : 0)));
  const cudaError_t e = launch_chained(f16 ? linear_fold_kernel<__half> : linear_fold_kernel<__nv_bfloat16>, grid,
                                       kFoldThreads, 0, cs, fp);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"

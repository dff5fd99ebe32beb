// Rows of an embedding table by id, and the table's gradient.
//
//   forward   y[t] = scale * table[ids[t]], zeros for an id below 0 (padding);
//   backward  dtable[v] = scale * the sum of dy[t] over the tokens with ids[t]
//             = v, summed in 32 bits in an order that the sorted tokens fix,
//             without atomics, so that two runs agree bit for bit.
//
// The backward sorts the tokens by id (stable, by digits of at most 9 bits from
// the lowest up), which puts the rows of one id next to each other, and then
// sums runs:
//   - the sorted tokens are cut into chunks of 16 to 128; a group of dim / 8
//     threads (8 columns a thread) walks a chunk's rows and writes a row of the
//     table at each change of id;
//   - a run that crosses into the next chunk belongs to the chunk it begins
//     in, unless it fills a whole chunk: such long runs (a few ids are most of
//     all tokens) leave a sum for each chunk in the workspace, and a join
//     kernel adds those in order;
//   - rows of the table that no token names are zeroed by further blocks of the
//     sorting and summing kernels, which know them by a bit a row that the first
//     pass set; every row of the table is so written once, and the sort, which
//     moves little, hides behind the zeros;
//   - up to 4096 tokens are sorted by one block of one launch.
#include <algorithm>
#include <cmath>

#include "layer.cuh"

namespace hstu {
namespace {

constexpr int kEmbedThreads = 256;
constexpr int kSortWarps = 16, kSortThreads = 32 * kSortWarps;
constexpr int kMaxDigitBits = 9, kMaxBins = 1 << kMaxDigitBits;
constexpr int kSortTiles = 152;  // at most one tile an SM
constexpr int kSeenBits = 10, kSeen = 1 << kSeenBits;
constexpr int kFillBytes = 1 << 17;     // of the table that a zeroing block looks after, about
constexpr int kFillMostRows = 1 << 13;  // of them (rows are 16 bytes at least)
// At most kJoinBlocks for long runs and for short ones: blocks that zero have the other half
// of the SMs from the start.
constexpr int kJoinThreads = 1024, kJoinBlocks = 76;
constexpr int kJoinCols = 512;  // of a joining block: 16 groups of threads share a long run
constexpr int kShortRun = 16;  // chunks of a run that one group of threads joins alone
// Header words: the long runs found, those of at most kShortRun chunks and the others.
constexpr int kHdrShort = 1, kHdrLong = 2;

// ------------------------------------------------------------------ forward

struct EmbedParams {
  const void* table;
  const void* ids;
  void* out;
  int32_t* header;  // null: bad ids are not reported
  int64_t vocab, tokens;
  uint64_t per_chunk;  // 2^32 / chunks, rounded up: u per_chunk / 2^32 is u / chunks for what a block has
  int32_t chunks;      // 8-column chunks of a row, 2^13 at most
  int32_t rows;        // rows of a block
  float scale;
};

// A block takes `rows` tokens' rows, U chunks a thread at a time; the ids of the next
// chunks are read while these are.
template <typename TT, typename T, typename ID, int U>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(const EmbedParams p) {
  chain();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(p.rows), p.tokens - t0));
  const uint32_t units = static_cast<uint32_t>(rows) * p.chunks;
  const ID* ids = static_cast<const ID*>(p.ids) + t0;
  const TT* table = static_cast<const TT*>(p.table);
  T* out = static_cast<T*>(p.out) + t0 * p.chunks * 8;
  ID next[U];
  auto read_ids = [&](uint32_t u0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = u0 + i * kEmbedThreads;
      next[i] = u < units ? ids[static_cast<uint32_t>(u * p.per_chunk >> 32)] : static_cast<ID>(-1);
    }
  };
  read_ids(threadIdx.x);
  for (uint32_t u0 = threadIdx.x; u0 < units; u0 += U * kEmbedThreads) {
    float f[U][8];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = u0 + i * kEmbedThreads, col = u - static_cast<uint32_t>(u * p.per_chunk >> 32) * p.chunks;
      const int64_t id = static_cast<int64_t>(next[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = 0.0f;
      if (id >= 0 && id < p.vocab) load8(table + (id * p.chunks + col) * 8, f[i]);
      else if (id >= p.vocab && p.header) atomicOr(p.header + kHdrErr, kErrInput);
    }
    read_ids(u0 + U * kEmbedThreads);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = u0 + i * kEmbedThreads;
      if (u >= units) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] *= p.scale;
      store8(out + static_cast<int64_t>(u) * 8, f[i]);
    }
  }
}

template <typename TT, typename T, typename ID>
cudaError_t launch_embed(EmbedParams p, cudaStream_t stream) {
  // Four chunks a thread at a time, and as many blocks as run at once, where that
  // fills the GPU; else one: a step's few rows are spread over as many SMs as they
  // have chunks for. (2^16 chunks a block at most, which per_chunk divides exactly.)
  const bool many = p.tokens * p.chunks >= int64_t{152} * 8 * kEmbedThreads * 4;
  const int64_t least = kEmbedThreads * (many ? 4 : 1) / p.chunks, even = many ? (p.tokens + 152 * 5 - 1) / (152 * 5) : 0;
  p.rows = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(std::max(least, even), (1 << 16) / p.chunks)));
  p.per_chunk = ((uint64_t{1} << 32) + p.chunks - 1) / p.chunks;
  const dim3 grid(static_cast<unsigned>((p.tokens + p.rows - 1) / p.rows));
  return launch_chained(many ? embed_kernel<TT, T, ID, 4> : embed_kernel<TT, T, ID, 1>, grid, kEmbedThreads, 0, stream, p);
}
template <typename ID>
cudaError_t launch_embed_typed(const EmbedParams& p, int table_dtype, int dtype, cudaStream_t stream) {
  using B = __nv_bfloat16;
  using H = __half;
  if (table_dtype == HSTU_DTYPE_F32)
    return dtype == HSTU_DTYPE_F16 ? launch_embed<float, H, ID>(p, stream) : launch_embed<float, B, ID>(p, stream);
  return dtype == HSTU_DTYPE_F16 ? launch_embed<H, H, ID>(p, stream) : launch_embed<B, B, ID>(p, stream);
}

// ------------------------------------------------------------------ zeroing

// Rows [row0, row1) of the table, those that no token names, as 16-byte units.
struct FillParams {
  void* table;
  const uint32_t* named;  // a bit a row; null: all rows
  int64_t row0, row1;
  uint64_t per_unit;  // 2^32 / units, rounded up: u per_unit / 2^32 is u / units for what a block has
  int32_t units;      // of a row, 2^14 at most
  int32_t rows;       // of a block
};
__host__ __device__ inline int64_t fill_blocks(const FillParams& p) {
  return p.row1 > p.row0 ? (p.row1 - p.row0 + p.rows - 1) / p.rows : 0;
}
__device__ __forceinline__ void fill_rows(const FillParams& p, int64_t block) {
  __shared__ uint32_t bits[kFillMostRows / 32 + 1];
  const int64_t v0 = p.row0 + block * p.rows, v1 = min(v0 + p.rows, p.row1), w0 = v0 >> 5;
  // The rows' bits first, so that no store waits for a load.
  for (int64_t w = w0 + threadIdx.x; w <= (v1 - 1) >> 5; w += blockDim.x) bits[w - w0] = p.named ? p.named[w] : 0u;
  __syncthreads();
  const uint32_t units = static_cast<uint32_t>(v1 - v0) * p.units, first = static_cast<uint32_t>(v0 & 31);
  uint4* base = static_cast<uint4*>(p.table) + v0 * p.units;
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 4
  for (uint32_t u = threadIdx.x; u < units; u += blockDim.x) {
    const uint32_t v = first + static_cast<uint32_t>(u * p.per_unit >> 32);
    if (((bits[v >> 5] >> (v & 31)) & 1u) == 0) base[u] = zero;
  }
}

// --------------------------------------------------------------------- sort

// One digit's pass over (id, token) pairs, from `ids` itself in the first.
struct SortParams {
  const void* ids;
  const uint32_t* key_in;
  const int32_t* val_in;
  uint32_t* key_out;
  int32_t* val_out;
  uint32_t* counts;  // (tiles, kMaxBins)
  uint32_t* named;   // first pass: a bit for each row of the table that a token names
  int32_t* header;   // null: bad ids are not reported
  int64_t vocab, n;
  int32_t tile;  // pairs of a tile, a multiple of kSortThreads
  int32_t tiles, shift, bits;
  FillParams fill;  // of the blocks behind the tiles'
};

// Padding and ids past the table sort behind it, as `vocab`.
template <typename ID, bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortParams& p, int64_t i) {
  if (!FIRST) return p.key_in[i];
  const int64_t id = static_cast<int64_t>(static_cast<const ID*>(p.ids)[i]);
  return id >= 0 && id < p.vocab ? static_cast<uint32_t>(id) : static_cast<uint32_t>(p.vocab);
}

// How often each digit occurs in each tile.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams p) {
  chain();
  if (static_cast<int>(blockIdx.x) >= p.tiles) return fill_rows(p.fill, blockIdx.x - p.tiles);
  __shared__ uint32_t count[kMaxBins];
  // Ids whose bit a thread of the block sets: the most frequent ids would otherwise
  // queue up at one word.
  __shared__ uint32_t seen[FIRST ? kSeen : 1];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) count[b] = 0;
  if (FIRST)
    for (int b = threadIdx.x; b < kSeen; b += kSortThreads) seen[b] = 0xffffffffu;
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.tile, i1 = min(i0 + p.tile, p.n);
#pragma unroll 4
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
    const uint32_t key = sort_key<ID, FIRST>(p, i);
    atomicAdd(&count[(key >> p.shift) & (bins - 1)], 1u);
    if (FIRST) {
      if (key < p.vocab) {
        if (atomicExch(&seen[(key * 2654435761u) >> (32 - kSeenBits)], key) == key) continue;
        atomicOr(p.named + (key >> 5), 1u << (key & 31));
      } else if (p.header && static_cast<int64_t>(static_cast<const ID*>(p.ids)[i]) >= 0)
        atomicOr(p.header + kHdrErr, kErrInput);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) p.counts[static_cast<int64_t>(blockIdx.x) * kMaxBins + b] = count[b];
}

// Moves each pair to its place: behind all pairs of a lower digit, those of its
// digit in earlier tiles, and those of its digit before it in the tile. A tile's
// warps own consecutive parts of it, so the order within a digit is kept.
template <typename ID, bool FIRST>
__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const SortParams p) {
  chain();
  if (static_cast<int>(blockIdx.x) >= p.tiles) return fill_rows(p.fill, blockIdx.x - p.tiles);
  __shared__ alignas(16) uint32_t place[kSortWarps][kMaxBins];
  __shared__ uint32_t warp_sum[kSortWarps];
  const int bins = 1 << p.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Digit b's pairs in all tiles and in those before this one. Groups of bins / 4 threads
  // take the tiles in turn, four digits a thread; thread b adds up the groups' sums.
  uint32_t total = 0, before = 0;
  {
    const int quads = max(bins / 4, 1), groups = min(kSortThreads / quads, kSortWarps / 2), g = threadIdx.x / quads;
    uint4 all = make_uint4(0, 0, 0, 0), low = all;
    if (g < groups) {
      const uint32_t* counts = p.counts + threadIdx.x % quads * 4;
#pragma unroll 8
      for (int t = g; t < p.tiles; t += groups) {
        const uint4 c = *reinterpret_cast<const uint4*>(counts + static_cast<int64_t>(t) * kMaxBins);
        all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
        if (t < static_cast<int>(blockIdx.x)) low.x += c.x, low.y += c.y, low.z += c.z, low.w += c.w;
      }
      *reinterpret_cast<uint4*>(&place[2 * g][threadIdx.x % quads * 4]) = all;
      *reinterpret_cast<uint4*>(&place[2 * g + 1][threadIdx.x % quads * 4]) = low;
    }
    __syncthreads();
    if (threadIdx.x < bins)
      for (int x = 0; x < groups; ++x) {
        total += place[2 * x][threadIdx.x];
        before += place[2 * x + 1][threadIdx.x];
      }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kSortWarps * kMaxBins; i += kSortThreads) (&place[0][0])[i] = 0;
  __syncthreads();
  const int part = p.tile / kSortWarps;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.tile + static_cast<int64_t>(warp) * part;
#pragma unroll 4
  for (int r = 0; r < part; r += 32) {
    const int64_t i = i0 + r + lane;
    if (i < p.n) atomicAdd(&place[warp][(sort_key<ID, FIRST>(p, i) >> p.shift) & (bins - 1)], 1u);
  }
  uint32_t sum = total;  // of digits up to this one
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += o;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  uint32_t at = sum - total + before;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  if (threadIdx.x < bins)
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = place[w][threadIdx.x];
      place[w][threadIdx.x] = at;
      at += c;
    }
  __syncthreads();
  auto val_at = [&](int64_t i) { return FIRST ? static_cast<int32_t>(i) : p.val_in[i]; };
  uint32_t next_key = i0 + lane < p.n ? sort_key<ID, FIRST>(p, i0 + lane) : 0;
  int32_t next_val = i0 + lane < p.n ? val_at(i0 + lane) : 0;
  for (int r = 0; r < part; r += 32) {
    const int64_t i = i0 + r + lane;
    const uint32_t live = __ballot_sync(0xffffffffu, i < p.n);
    const uint32_t key = next_key;
    const int32_t val = next_val;
    if (i + 32 < p.n && r + 32 < part) {
      next_key = sort_key<ID, FIRST>(p, i + 32);
      next_val = val_at(i + 32);
    }
    if (i < p.n) {
      const uint32_t digit = (key >> p.shift) & (bins - 1);
      const uint32_t same = __match_any_sync(live, digit);
      const uint32_t to = place[warp][digit] + __popc(same & ((1u << lane) - 1u));
      __syncwarp(live);
      if (lane == 31 - __clz(same)) place[warp][digit] = to + 1;
      p.key_out[to] = key;
      p.val_out[to] = val;
    }
    __syncwarp();
  }
}

// Few tokens in one launch (1889 tokens forward and backward take 20 us, 29 us with two
// launches a digit): a block keeps its pairs in registers, kBlockRounds a thread, and
// turns them over in shared memory once a digit. A pair's place is that of its digit and
// warp plus the number of the warp's pairs of the digit before it. The other blocks zero
// the table, named rows too, which are few and are written after.
constexpr int kBlockThreads = 1024, kBlockWarps = kBlockThreads / 32, kBlockRounds = 4;
constexpr int kBlockTokens = kBlockThreads * kBlockRounds;
constexpr int kBlockSmem = kBlockTokens * 8 + kBlockWarps * kMaxBins * 2;
template <typename ID>
__global__ void __launch_bounds__(kBlockThreads) sort_block_kernel(const SortParams p, int passes) {
  chain();
  if (blockIdx.x > 0) return fill_rows(p.fill, blockIdx.x - 1);
  extern __shared__ uint4 sort_smem[];
  uint16_t(*place)[kMaxBins] = reinterpret_cast<uint16_t(*)[kMaxBins]>(sort_smem);
  uint2* pairs = reinterpret_cast<uint2*>(sort_smem + kBlockWarps * kMaxBins * 2 / 16);
  __shared__ uint32_t warp_sum[kBlockWarps];
  const int n = static_cast<int>(p.n), rounds = (n + kBlockThreads - 1) / kBlockThreads;
  const int bins = 1 << p.bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i0 = warp * rounds * 32 + lane;
  if (threadIdx.x < kHdrWords) p.header[threadIdx.x] = 0;
  uint32_t key[kBlockRounds];
  int32_t val[kBlockRounds];
  bool past = false;  // an id past the table
#pragma unroll
  for (int r = 0; r < kBlockRounds; ++r) {
    const int i = i0 + 32 * r;
    val[r] = i;
    key[r] = 0;
    if (r < rounds && i < n) {
      key[r] = sort_key<ID, true>(p, i);
      past |= key[r] == p.vocab && static_cast<int64_t>(static_cast<const ID*>(p.ids)[i]) >= 0;
    }
  }
  for (int s = 0; s < passes; ++s) {
    for (int i = threadIdx.x; i < kBlockWarps * kMaxBins * 2 / 16; i += kBlockThreads) sort_smem[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    uint32_t digit[kBlockRounds], nth[kBlockRounds];
#pragma unroll
    for (int r = 0; r < kBlockRounds; ++r) {
      const bool mine = r < rounds && i0 + 32 * r < n;
      const uint32_t live = __ballot_sync(0xffffffffu, mine);
      digit[r] = nth[r] = 0;
      if (mine) {
        digit[r] = (key[r] >> (s * p.bits)) & (bins - 1);
        const uint32_t same = __match_any_sync(live, digit[r]);
        nth[r] = place[warp][digit[r]] + __popc(same & ((1u << lane) - 1u));
        __syncwarp(live);
        if (lane == 31 - __clz(same)) place[warp][digit[r]] = static_cast<uint16_t>(nth[r] + 1);
      }
      __syncwarp();
    }
    __syncthreads();
    // Thread b: where digit b's pairs of each warp begin.
    uint32_t total = 0;
    if (threadIdx.x < bins)
#pragma unroll
      for (int w = 0; w < kBlockWarps; ++w) total += place[w][threadIdx.x];
    uint32_t sum = total;  // of digits up to this one
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    uint32_t at = sum - total;
    if (threadIdx.x < bins) {
      for (int w = 0; w < warp; ++w) at += warp_sum[w];
#pragma unroll
      for (int w = 0; w < kBlockWarps; ++w) {
        const uint32_t c = place[w][threadIdx.x];
        place[w][threadIdx.x] = static_cast<uint16_t>(at);
        at += c;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kBlockRounds; ++r)
      if (r < rounds && i0 + 32 * r < n) pairs[place[warp][digit[r]] + nth[r]] = make_uint2(key[r], static_cast<uint32_t>(val[r]));
    __syncthreads();
    if (s + 1 < passes)
#pragma unroll
      for (int r = 0; r < kBlockRounds; ++r)
        if (r < rounds && i0 + 32 * r < n) {
          const uint2 q = pairs[i0 + 32 * r];
          key[r] = q.x;
          val[r] = static_cast<int32_t>(q.y);
        }
  }
  for (int i = threadIdx.x; i < n; i += kBlockThreads) {
    const uint2 q = pairs[i];
    p.key_out[i] = q.x;
    p.val_out[i] = static_cast<int32_t>(q.y);
  }
  if (past) atomicOr(p.header + kHdrErr, kErrInput);
}

// ----------------------------------------------------------------- backward

struct SumParams {
  const void* dy;
  int64_t dy_stride;
  const uint32_t* key;  // sorted ids
  const int32_t* val;   // their tokens
  void* dtable;
  float* part;  // (chunks, 2, dim): sums of long runs' chunks; [0] of a run from an earlier chunk, [1] of one that begins
  int32_t* header;
  int32_t* runs;  // first whole chunks: of short runs from the front, of others from the back
  int64_t n, vocab;
  int32_t chunk, chunks, dim, accumulate;
  int32_t groups;      // chunks of a summing block
  int32_t long_blocks, short_blocks;  // of the join, for the runs of either kind
  int32_t sum_blocks;  // blocks that sum, spread evenly among those that zero
  float scale;
  FillParams fill;
};

template <typename G>
__device__ __forceinline__ void put_row(const SumParams& p, int64_t row, int col, float (&acc)[8]) {
  G* dst = static_cast<G*>(p.dtable) + row * p.dim + col;
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] *= p.scale;
  if (p.accumulate) {
    float old[8];
    load8(dst, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += old[e];
  }
  store8(dst, acc);
}

template <typename T, typename G>
__global__ void __launch_bounds__(kEmbedThreads) embed_sum_kernel(const SumParams p) {
  chain();
  const int64_t summed = static_cast<int64_t>(blockIdx.x) * p.sum_blocks / gridDim.x;  // summing blocks before this one
  if ((static_cast<int64_t>(blockIdx.x) + 1) * p.sum_blocks / gridDim.x == summed) {
    if (blockIdx.y == 0) fill_rows(p.fill, blockIdx.x - summed);
    return;
  }
  const int col0 = blockIdx.y * kEmbedThreads * 8;
  const int group = min(kEmbedThreads, (p.dim - col0) / 8);  // threads of a row
  const int groups = p.groups, g = threadIdx.x / group;
  const int col = col0 + (threadIdx.x % group) * 8;
  if (g >= groups) return;
  const int64_t c = summed * groups + g;
  if (c >= p.chunks) return;
  // The ids at the chunk's ends and its neighbours', all read at once: kNoId where there
  // is none.
  constexpr uint32_t kNoId = 0xffffffffu;
  const int64_t i0 = c * p.chunk, end = min(i0 + p.chunk, p.n), far = i0 + static_cast<int64_t>(kShortRun) * p.chunk;
  const uint32_t first = p.key[i0], last = p.key[end - 1];
  const uint32_t before = c > 0 ? p.key[i0 - 1] : kNoId, before_first = c > 0 ? p.key[i0 - p.chunk] : kNoId;
  const uint32_t after = end < p.n ? p.key[end] : kNoId;
  const uint32_t after_last = end < p.n ? p.key[min(end + p.chunk, p.n) - 1] : kNoId;
  const uint32_t far_first = far < p.n ? p.key[far] : kNoId;
  if (first >= p.vocab) return;
  const bool whole = first == last, from_before = before == first;
  // How many of the ids from `at` on, a chunk's at most, are `id`.
  auto run_of = [&](int64_t at, int64_t limit, uint32_t id) {
    int n = 0;
    for (int part = 0; part < p.chunk; part += 16) {
      int same = 0;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int64_t x = at + part + u;
        same += x < limit && p.key[x] == id;
      }
      n += same;
      if (same < 16) break;
    }
    return n;
  };
  int64_t i = i0, i1 = end;
  // The run that comes from the chunk before: the whole of a chunk, or the end
  // of a long run (one that fills the chunk before), is a partial sum;
  // otherwise that chunk sums it.
  const bool long_before = from_before && before_first == first;
  const bool head_part = whole || long_before;
  if (from_before && !head_part) i += run_of(i0, end, first);
  // The run that goes on into the next chunk: long if that chunk is full of it, else it is
  // summed here to its end.
  const bool goes_on = !whole && after == last && last < p.vocab, tail_part = goes_on && after_last == last;
  if (goes_on && !tail_part) i1 += run_of(end, p.n, last);
  // A whole chunk whose run is no longer than it: an ordinary row.
  const bool alone = whole && !from_before && after != first;
  // The first whole chunk of a run lists it for the join. (In whatever order: each
  // run is added up by itself.)
  if (whole && !alone && !long_before && blockIdx.y == 0 && threadIdx.x % group == 0) {
    const bool brief = far_first != first;
    const int at = atomicAdd(p.header + (brief ? kHdrShort : kHdrLong), 1);
    p.runs[brief ? at : p.chunks - 1 - at] = static_cast<int32_t>(c);
  }
  const T* dy = static_cast<const T*>(p.dy) + col;
  float acc[8] = {};
  uint32_t cur = i < i1 ? p.key[i] : 0xffffffffu;
  auto flush = [&](uint32_t row) {
    if (row >= p.vocab) return;
    if (!alone && head_part && row == first) {
      store8(p.part + (c * 2) * p.dim + col, acc);
    } else if (tail_part && row == last) {
      store8(p.part + (c * 2 + 1) * p.dim + col, acc);
    } else {
      put_row<G>(p, row, col, acc);
    }
  };
  // Four rows at a time; their ids and tokens are read while the four before are added.
  constexpr int kAhead = 4;
  uint32_t key[kAhead], next_key[kAhead];
  int32_t val[kAhead], next_val[kAhead];
  auto read_ids = [&](int64_t at, uint32_t (&k)[kAhead], int32_t (&t)[kAhead]) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      k[a] = at + a < i1 ? p.key[at + a] : 0xffffffffu;
      t[a] = at + a < i1 ? p.val[at + a] : 0;
    }
  };
  read_ids(i, key, val);
  while (i < i1) {
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (key[a] < p.vocab) v[a] = *reinterpret_cast<const uint4*>(dy + static_cast<int64_t>(val[a]) * p.dy_stride);
    read_ids(i + kAhead, next_key, next_val);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (key[a] != cur) {  // past the last token too
        flush(cur);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        cur = key[a];
      }
      if (key[a] >= p.vocab) return;  // padding sorts last
      float f[8];
      unpack8<T>(v[a], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[e];
    }
    i += kAhead;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      key[a] = next_key[a];
      val[a] = next_val[a];
    }
  }
  flush(cur);
}

// Adds up the chunks of each long run: the end of the chunk before its first
// whole one, the whole ones, and the beginning of the chunk behind. A run of a
// few chunks is one group's, a longer one all groups': they take consecutive slices
// of it, which are added in order.
template <typename G>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(const SumParams p) {
  chain();
  const int joining = p.long_blocks + p.short_blocks;
  if (static_cast<int>(blockIdx.x) >= joining) {
    if (blockIdx.y == 0) fill_rows(p.fill, blockIdx.x - joining);
    return;
  }
  __shared__ float slice[kJoinThreads][8];
  const int brief = p.header[kHdrShort], large = p.header[kHdrLong];
  const int col0 = blockIdx.y * kJoinCols;
  const int group = min(kJoinCols, p.dim - col0) / 8;
  const int groups = kJoinThreads / group, g = threadIdx.x / group;
  const int col = col0 + (threadIdx.x % group) * 8;
  // The sum of chunks [a, b) of a run; of the end of the chunk before too with `before`.
  auto sum_of = [&](int64_t a, int64_t b, bool before, float (&acc)[8]) {
    if (before) load8(p.part + ((a - 1) * 2 + 1) * p.dim + col, acc);
#pragma unroll 8
    for (int64_t x = a; x < b; ++x) {
      float f[8];
      load8(p.part + x * 2 * p.dim + col, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[e];
    }
  };
  auto from_before = [&](int64_t c, uint32_t key) { return c > 0 && p.key[c * p.chunk - 1] == key; };
  if (g < groups)
    for (int k = (static_cast<int>(blockIdx.x) - p.long_blocks) * groups + g; k >= 0 && k < brief; k += p.short_blocks * groups) {
      const int64_t c = p.runs[k];
      const uint32_t key = p.key[c * p.chunk];
      int parts = 1;
      bool on = true;
#pragma unroll
      for (int x = 1; x < kShortRun; ++x) {
        on = c + x < p.chunks && p.key[(c + x) * p.chunk] == key && on;
        parts += on;
      }
      float acc[8] = {};
      sum_of(c, c + parts, from_before(c, key), acc);
      put_row<G>(p, key, col, acc);
    }
  if (static_cast<int>(blockIdx.x) >= p.long_blocks) return;
  for (int k = blockIdx.x; k < large; k += p.long_blocks) {
    const int64_t c = p.runs[p.chunks - 1 - k];
    const uint32_t key = p.key[c * p.chunk];
    // The last chunk that begins with the id: all threads look, at a step that
    // shrinks a thousandfold.
    int64_t last = c;
    for (int64_t span = p.chunks - c; span > 1;) {
      const int64_t step = (span - 1 + kJoinThreads - 1) / kJoinThreads, x = (threadIdx.x + 1) * step;
      const int hits = __syncthreads_count(x < span && p.key[(last + x) * p.chunk] == key);
      last += hits * step;
      span = min(step, span - hits * step);
    }
    const int64_t parts = last - c + 1, per = (parts + groups - 1) / groups;
    float acc[8] = {};
    if (g < groups) {
      const int64_t a = c + min(g * per, parts), b = c + min((g + 1) * per, parts);
      sum_of(a, b, g == 0 && from_before(c, key), acc);
#pragma unroll
      for (int e = 0; e < 8; ++e) slice[threadIdx.x][e] = acc[e];
    }
    __syncthreads();
    if (g == 0) {
      for (int x = 1; x < groups; ++x)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += slice[x * group + threadIdx.x][e];
      put_row<G>(p, key, col, acc);
    }
    __syncthreads();
  }
}

// No tokens: every row is zero.
__global__ void __launch_bounds__(kEmbedThreads) embed_zero_kernel(const FillParams p) {
  chain();
  fill_rows(p, blockIdx.x);
}

// A chunk's tokens: enough chunks to fill the GPU (2048 threads on each of 152 SMs), 16
// to 128.
int sum_chunk(int64_t n, int dim) {
  const int64_t want = n * (dim / 8) / (152 * 2048);
  int c = 16;
  while (c < 128 && 2 * c <= want) c *= 2;
  return c;
}

// The most chunks of up to n tokens, so that a workspace serves calls of fewer.
int64_t most_chunks(int64_t n, int dim) {
  int64_t most = 0;
  for (int c = 16; c <= sum_chunk(n, dim); c *= 2) {
    const int64_t last = c < 128 ? std::min(n, (int64_t{2} * c * 152 * 2048 - 1) / (dim / 8)) : n;  // with chunks of c
    most = std::max(most, (last + c - 1) / c);
  }
  return most;
}

// Workspace: a 256-byte header (error word), a bit a row of the table, the two
// buffers of (id, token), the digits' counts, and the long runs' list and sums.
struct EmbedLayout {
  size_t named = 0, key[2] = {}, val[2] = {}, counts = 0, runs = 0, part = 0, total = 0;
};
EmbedLayout embed_layout(int64_t n, int64_t vocab, int dim) {
  EmbedLayout l;
  l.named = kHdrWords * 4;
  size_t at = l.named + align_up(static_cast<size_t>((vocab + 31) / 32) * 4, 256);
  for (int i = 0; i < 2; ++i) {
    l.key[i] = at;
    at += align_up(static_cast<size_t>(n) * 4, 256);
    l.val[i] = at;
    at += align_up(static_cast<size_t>(n) * 4, 256);
  }
  l.counts = at;
  at += static_cast<size_t>(kSortTiles) * kMaxBins * 4;
  const size_t chunks = static_cast<size_t>(most_chunks(n, dim));
  l.runs = at;
  at += align_up(chunks * 4, 256);
  l.part = at;
  at += align_up(chunks * 2 * dim * 4, 256);
  l.total = at;
  return l;
}

// Takes `part` of `parts` of the table's rows from those still to be zeroed.
FillParams fill_share(FillParams& rest, int64_t rows, int part, int parts) {
  FillParams f = rest;
  f.row1 = std::min(f.row0 + rows * part / parts, rest.row1);
  rest.row0 = f.row1;
  return f;
}

// The launches that follow the first zero rows on the side: a move four parts, a
// count, which is about half as long, two; the summing kernel, which moves as much
// itself, and the join, which mostly waits, three each. (81920 tokens, 200003 rows of 512:
// sort, sum and join take 65 us without zeros, the zeros alone 53 us.)
// Leaves the rows still to be zeroed in `fill`.
template <typename ID>
cudaError_t launch_sort(SortParams p, FillParams& fill, uint8_t* base, const EmbedLayout& l, int& last,
                        cudaStream_t stream) {
  const int64_t all = fill.row1 - fill.row0;
  int bits = 1;
  while ((p.vocab >> bits) != 0) ++bits;  // of the largest key, vocab
  const int passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.bits = (bits + passes - 1) / passes;
  if (p.n <= kBlockTokens) {
    p.key_out = reinterpret_cast<uint32_t*>(base + l.key[0]);
    p.val_out = reinterpret_cast<int32_t*>(base + l.val[0]);
    last = 0;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = ensure_smem_limit(sort_block_kernel<ID>, kBlockSmem, configured);
    if (e != cudaSuccess) return e;
    p.fill = fill;
    p.fill.named = nullptr;
    fill.row0 = fill.row1;
    return launch_chained(sort_block_kernel<ID>, dim3(static_cast<unsigned>(1 + fill_blocks(p.fill))), kBlockThreads,
                          kBlockSmem, stream, p, passes);
  }
  const int parts = 4 * passes + 2 * (passes - 1) + 6;
  const int64_t rounds = (p.n + int64_t{kSortTiles} * kSortThreads - 1) / (int64_t{kSortTiles} * kSortThreads);
  p.tile = static_cast<int32_t>(rounds * kSortThreads);
  p.tiles = static_cast<int32_t>((p.n + p.tile - 1) / p.tile);
  for (int s = 0; s < passes; ++s) {
    p.shift = s * p.bits;
    p.key_in = reinterpret_cast<const uint32_t*>(base + l.key[s & 1]);
    p.val_in = reinterpret_cast<const int32_t*>(base + l.val[s & 1]);
    p.key_out = reinterpret_cast<uint32_t*>(base + l.key[(s + 1) & 1]);
    p.val_out = reinterpret_cast<int32_t*>(base + l.val[(s + 1) & 1]);
    p.fill = fill_share(fill, all, s == 0 ? 0 : 2, parts);  // (the first launch sets the rows' bits)
    cudaError_t e = launch_chained(s == 0 ? sort_count_kernel<ID, true> : sort_count_kernel<ID, false>,
                                   dim3(static_cast<unsigned>(p.tiles + fill_blocks(p.fill))), kSortThreads, 0, stream, p);
    if (e != cudaSuccess) return e;
    p.fill = fill_share(fill, all, 4, parts);
    e = launch_chained(s == 0 ? sort_move_kernel<ID, true> : sort_move_kernel<ID, false>,
                       dim3(static_cast<unsigned>(p.tiles + fill_blocks(p.fill))), kSortThreads, 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  last = passes & 1;
  return cudaSuccess;
}

// The rows of the table still to be zeroed (`fill`) are shared with the join.
template <typename T, typename G>
cudaError_t launch_sum(SumParams p, FillParams fill, cudaStream_t stream) {
  const int widest = p.dim < kEmbedThreads * 8 ? p.dim : kEmbedThreads * 8;
  // As many chunks as fit a block, and no more threads than they need (a row of 1128
  // columns takes 141: one chunk, 160 threads).
  p.groups = kEmbedThreads / (widest / 8);
  const int threads = (p.groups * (widest / 8) + 31) / 32 * 32;
  const unsigned ny = (p.dim + kEmbedThreads * 8 - 1) / (kEmbedThreads * 8);
  p.sum_blocks = (p.chunks + p.groups - 1) / p.groups;
  const bool join = p.chunks > 1;  // a chunk alone has no runs into others
  p.fill = fill_share(fill, fill.row1 - fill.row0, 1, join ? 2 : 1);
  cudaError_t e = launch_chained(embed_sum_kernel<T, G>, dim3(static_cast<unsigned>(p.sum_blocks + fill_blocks(p.fill)), ny),
                                 threads, 0, stream, p);
  if (e != cudaSuccess || !join) return e;
  p.fill = fill;
  // No more blocks than there can be runs.
  const int join_groups = kJoinThreads / (std::min(kJoinCols, p.dim) / 8);
  p.long_blocks = std::min(kJoinBlocks, (p.chunks + kShortRun - 1) / kShortRun);
  p.short_blocks = std::min(kJoinBlocks, (p.chunks + join_groups - 1) / join_groups);
  return launch_chained(embed_join_kernel<G>,
                        dim3(static_cast<unsigned>(p.long_blocks + p.short_blocks + fill_blocks(fill)),
                             (p.dim + kJoinCols - 1) / kJoinCols),
                        kJoinThreads, 0, stream, p);
}
template <typename T>
cudaError_t launch_sum_typed(const SumParams& p, const FillParams& fill, int grad_dtype, cudaStream_t stream) {
  return grad_dtype == HSTU_DTYPE_F32 ? launch_sum<T, float>(p, fill, stream) : launch_sum<T, T>(p, fill, stream);
}

hstu_status_t embed_checks(int64_t tokens, int64_t vocab, int dim) {
  if (tokens < 0 || tokens > INT32_MAX || vocab < 1 || vocab >= INT32_MAX || dim < 1) return HSTU_ERR_INVALID_ARG;
  if (dim % 8 != 0 || dim > 65536) return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}
bool embed_types_ok(int dtype, int wide, int id_bytes) {
  return row_dtype_ok(dtype) && (wide == dtype || wide == HSTU_DTYPE_F32) && (id_bytes == 4 || id_bytes == 8);
}

}  // namespace
}  // namespace hstu

extern "C" {

HSTU_API hstu_status_t hstu_attn_embed(const void* table, int32_t table_dtype, int64_t vocab, int32_t dim,
                                       const void* ids, int32_t id_bytes, int64_t tokens, float scale, void* out,
                                       int32_t dtype, void* ws, size_t ws_bytes, void* stream) {
  using namespace hstu;
  const hstu_status_t st = embed_checks(tokens, vocab, dim);
  if (st != HSTU_OK) return st;
  if (!embed_types_ok(dtype, table_dtype, id_bytes)) return HSTU_ERR_UNSUPPORTED;
  // The kernel scales the zeros of padding too. (A choice between scales there costs registers, and with
  // them a block of an SM: 81920 rows of 512 in 42 us, not 30.)
  if (!std::isfinite(scale)) return HSTU_ERR_INVALID_ARG;
  if (ws && (!aligned_to(ws, 256) || ws_bytes < kHdrWords * 4)) return HSTU_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (tokens > 0) {
    if (!aligned_to(table, table_dtype == HSTU_DTYPE_F32 ? 32 : 16) || !aligned_to(out, 16) || !aligned_to(ids, id_bytes)) return HSTU_ERR_INVALID_ARG;
    const int64_t written = tokens * dim * 2;
    if (ranges_meet(out, written, table, vocab * dim * (table_dtype == HSTU_DTYPE_F32 ? 4 : 2)) ||
        ranges_meet(out, written, ids, tokens * id_bytes))
      return HSTU_ERR_INVALID_ARG;
  }
  if (ws && cudaMemsetAsync(ws, 0, kHdrWords * 4, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  if (tokens == 0) return HSTU_OK;
  EmbedParams p{};
  p.table = table;
  p.ids = ids;
  p.out = out;
  p.header = static_cast<int32_t*>(ws);
  p.vocab = vocab;
  p.tokens = tokens;
  p.chunks = dim / 8;
  p.scale = scale;
  const cudaError_t e = id_bytes == 8 ? launch_embed_typed<int64_t>(p, table_dtype, dtype, cs)
                                      : launch_embed_typed<int32_t>(p, table_dtype, dtype, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

HSTU_API size_t hstu_attn_embed_workspace_size(int64_t tokens, int64_t vocab, int32_t dim) {
  return hstu::embed_checks(tokens, vocab, dim) == HSTU_OK ? hstu::embed_layout(tokens, vocab, dim).total : 0;
}

HSTU_API hstu_status_t hstu_attn_embed_bwd(const void* dy, int64_t dy_stride, int32_t dtype, const void* ids,
                                           int32_t id_bytes, int64_t tokens, float scale, void* dtable,
                                           int32_t grad_dtype, int64_t vocab, int32_t dim, int32_t accumulate, void* ws,
                                           size_t ws_bytes, void* stream) {
  using namespace hstu;
  const hstu_status_t st = embed_checks(tokens, vocab, dim);
  if (st != HSTU_OK) return st;
  if (!embed_types_ok(dtype, grad_dtype, id_bytes)) return HSTU_ERR_UNSUPPORTED;
  if (accumulate != 0 && accumulate != 1) return HSTU_ERR_INVALID_ARG;
  if (accumulate && grad_dtype != HSTU_DTYPE_F32) return HSTU_ERR_UNSUPPORTED;
  if (!aligned_to(dtable, grad_dtype == HSTU_DTYPE_F32 ? 32 : 16)) return HSTU_ERR_INVALID_ARG;
  if (tokens > 0) {
    if (!rows_ok(dy, dy_stride, 1, dim) || !aligned_to(ids, id_bytes)) return HSTU_ERR_INVALID_ARG;
    const int64_t bytes = vocab * dim * (grad_dtype == HSTU_DTYPE_F32 ? 4 : 2);
    if (ranges_meet(dtable, bytes, dy, ((tokens - 1) * dy_stride + dim) * 2) ||
        ranges_meet(dtable, bytes, ids, tokens * id_bytes))
      return HSTU_ERR_INVALID_ARG;
  }
  const EmbedLayout l = embed_layout(tokens, vocab, dim);
  if (!aligned_to(ws, 256) || ws_bytes < l.total) return HSTU_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  // The error word and the bits of the rows. (A sort in one block needs no bits.)
  if ((tokens == 0 || tokens > kBlockTokens) && cudaMemsetAsync(base, 0, l.key[0], cs) != cudaSuccess)
    return HSTU_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  FillParams fill{};
  fill.table = dtable;
  fill.named = reinterpret_cast<const uint32_t*>(base + l.named);
  fill.row1 = accumulate ? 0 : vocab;
  fill.units = dim / (grad_dtype == HSTU_DTYPE_F32 ? 4 : 8);
  fill.per_unit = ((uint64_t{1} << 32) + fill.units - 1) / fill.units;
  fill.rows = std::max(1, std::min(kFillBytes / (16 * fill.units), kFillMostRows));
  if (tokens == 0) {
    if (accumulate) return HSTU_OK;
    e = launch_chained(embed_zero_kernel, dim3(static_cast<unsigned>(fill_blocks(fill))), kEmbedThreads, 0, cs, fill);
    return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
  }
  SortParams sp{};
  sp.ids = ids;
  sp.counts = reinterpret_cast<uint32_t*>(base + l.counts);
  sp.named = reinterpret_cast<uint32_t*>(base + l.named);
  sp.header = reinterpret_cast<int32_t*>(base);
  sp.vocab = vocab;
  sp.n = tokens;
  int last = 0;
  e = id_bytes == 8 ? launch_sort<int64_t>(sp, fill, base, l, last, cs)
                    : launch_sort<int32_t>(sp, fill, base, l, last, cs);
  if (e != cudaSuccess) return HSTU_ERR_CUDA;
  SumParams p{};
  p.dy = dy;
  p.dy_stride = dy_stride;
  p.key = reinterpret_cast<const uint32_t*>(base + l.key[last]);
  p.val = reinterpret_cast<const int32_t*>(base + l.val[last]);
  p.dtable = dtable;
  p.part = reinterpret_cast<float*>(base + l.part);
  p.header = reinterpret_cast<int32_t*>(base);
  p.runs = reinterpret_cast<int32_t*>(base + l.runs);
  p.n = tokens;
  p.vocab = vocab;
  p.dim = dim;
  p.chunk = sum_chunk(tokens, dim);
  p.chunks = static_cast<int32_t>((tokens + p.chunk - 1) / p.chunk);
  p.accumulate = accumulate;
  p.scale = scale;
  e = dtype == HSTU_DTYPE_F16 ? launch_sum_typed<__half>(p, fill, grad_dtype, cs)
                              : launch_sum_typed<__nv_bfloat16>(p, fill, grad_dtype, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"

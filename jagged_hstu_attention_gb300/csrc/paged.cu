// Entry points of the paged attention (declared in include/hstu_attn.h):
// argument checks, the split of the cache's length, workspace, dispatch.
#include <algorithm>

#include "paged_many.cuh"

namespace hstu {

// The split of the cache's length. It follows from the arguments alone, so
// that the workspace and the order of the sums are the same on every device.
//   - As many keys as leave 2400 CTAs (eight waves of two an SM) at the longest
//     length, which balances ragged lengths, from 512 to 4096.
//   - With more than 8 candidates a sequence on average in paged_kernel, 1024 keys at
//     the least, which paged_split_keys cuts to a half or a quarter where a sequence
//     has many: 64 users of 512 to 2048 rows and 0 to 48 candidates took 64 us so and
//     72 us with 512 keys for all. With fewer the short splits that no sequence uses
//     would cost more than they give.
//   - paged_many_kernel (widths of 128, bf16 or 8-bit pages, more than 16 candidates
//     on average, N above 256; its header has both kernels' times) takes 60 us of
//     them with 512 keys at the least, 61 with 1024 and 58 with 2048; 16 users of
//     20000 rows 176 with 512.
struct PagedLayout {
  int split = 0, nsplit = 0;
  bool tensor = false, shorter = false;
  size_t states = 0, partial = 0, total = 0;
};
static PagedLayout paged_layout(const CacheView& c, const hstu_cache_t* cache, int batch, int64_t num_cand,
                                int max_seqlen) {
  constexpr int64_t kCtas = 2400;
  PagedLayout l;
  l.tensor = c.dim == kManyDim && c.dim_v == kManyDim && (cache->e4m3 || cache->dtype != HSTU_DTYPE_F16) &&
             num_cand > 16 * static_cast<int64_t>(batch) && max_seqlen > 256;
  l.shorter = !l.tensor && num_cand > 8 * static_cast<int64_t>(batch);
  const int64_t want = static_cast<int64_t>(max_seqlen) * batch * c.heads / kCtas;
  l.split = static_cast<int>(
      std::min<int64_t>(kPagedMaxSplit, std::max<int64_t>(l.shorter ? 1024 : 512, (want + 255) / 256 * 256)));
  const int least = l.shorter ? l.split / paged_slice(kPagedPass) : l.split;
  l.nsplit = (max_seqlen + least - 1) / least;
  l.states = l.partial = l.total = kHdrWords * 4;
  if (l.nsplit > 1) {
    l.partial = l.states + align_up(static_cast<size_t>(batch) * c.heads * l.nsplit * 4, 256);
    l.total = l.partial + align_up(static_cast<size_t>(num_cand) * c.heads * l.nsplit * c.dim_v * 4, 256);
  }
  // paged_kernel's shorter splits can take more room for fewer candidates: a
  // workspace serves every call with as many or fewer.
  if (l.tensor)
    l.total = std::max(l.total, paged_layout(c, cache, batch, 16 * static_cast<int64_t>(batch), max_seqlen).total);
  return l;
}

static hstu_status_t check_paged(const hstu_cache_t* cache, int32_t batch, int64_t num_cand, int32_t max_seqlen,
                                 CacheView* view) {
  const hstu_status_t st = check_cache(cache, view);
  if (st != HSTU_OK) return st;
  if (batch < 1 || num_cand < 0 || num_cand > INT32_MAX || max_seqlen < 1) return HSTU_ERR_INVALID_ARG;
  if (max_seqlen > (1 << 24)) return HSTU_ERR_UNSUPPORTED;
  const PagedLayout l = paged_layout(*view, cache, batch, num_cand, max_seqlen);
  const int64_t bh = static_cast<int64_t>(batch) * view->heads;
  if (bh > INT32_MAX / l.nsplit || num_cand * view->heads > INT32_MAX) return HSTU_ERR_UNSUPPORTED;  // CTAs of a launch
  return HSTU_OK;
}

}  // namespace hstu

extern "C" {

HSTU_API size_t hstu_attn_paged_workspace_size(const hstu_cache_t* cache, int32_t batch, int64_t num_candidates,
                                               int32_t max_seqlen) {
  hstu::CacheView view;
  if (hstu::check_paged(cache, batch, num_candidates, max_seqlen, &view) != HSTU_OK) return 0;
  return hstu::paged_layout(view, cache, batch, num_candidates, max_seqlen).total;
}

HSTU_API hstu_status_t hstu_attn_fwd_paged(const void* q_c, int64_t q_stride, void* o_c, const hstu_cache_t* cache,
                                           const int32_t* cache_lens, int32_t batch, const int32_t* page_table,
                                           int32_t max_pages, const int32_t* cand_offsets, int64_t num_candidates,
                                           const int32_t* func_c, int32_t nfunc, int32_t max_seqlen, float alpha,
                                           void* ws, size_t ws_bytes, uint32_t flags, void* stream) {
  hstu::PagedParams p{};
  const hstu_status_t st = hstu::check_paged(cache, batch, num_candidates, max_seqlen, &p.cache);
  if (st != HSTU_OK) return st;
  if (func_c && !hstu_attn_nfunc_supported(nfunc)) return HSTU_ERR_UNSUPPORTED;
  if (max_pages < 1 || !(alpha == alpha) || (!cand_offsets && num_candidates != batch)) return HSTU_ERR_INVALID_ARG;
  const auto bad4 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 4 != 0; };
  if (!cache_lens || !page_table || bad4(cache_lens) || bad4(page_table) || bad4(cand_offsets) || bad4(func_c))
    return HSTU_ERR_INVALID_ARG;
  if (num_candidates > 0 && (!hstu::rows_ok(q_c, q_stride, p.cache.heads, p.cache.dim) || !o_c ||
                             reinterpret_cast<uintptr_t>(o_c) % 16 != 0))
    return HSTU_ERR_INVALID_ARG;
  const int64_t q_row = 2ll * p.cache.heads * p.cache.dim, o_row = 2ll * p.cache.heads * p.cache.dim_v;
  if (hstu::rows_meet(o_c, o_row, o_row, q_c, 2 * q_stride, q_row, num_candidates)) return HSTU_ERR_INVALID_ARG;
  const bool half = cache->dtype == HSTU_DTYPE_F16;
  const hstu::PagedLayout l = hstu::paged_layout(p.cache, cache, batch, num_candidates, max_seqlen);
  const bool report = !(flags & HSTU_FLAG_NO_STATUS);
  if (!ws && (l.nsplit > 1 || report)) return HSTU_ERR_WORKSPACE;
  if (ws && (reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < l.total)) return HSTU_ERR_WORKSPACE;
  uint8_t* base = static_cast<uint8_t*>(ws);
  p.q = q_c;
  p.o = o_c;
  p.q_stride = q_stride;
  p.lens = cache_lens;
  p.page_table = page_table;
  p.cand_offsets = cand_offsets;
  p.func = func_c;
  p.partial = reinterpret_cast<float*>(base + l.partial);
  p.header = report ? reinterpret_cast<int32_t*>(base) : nullptr;
  p.states = reinterpret_cast<int32_t*>(base + l.states);
  p.batch = batch;
  p.max_pages = max_pages;
  p.num_cand = static_cast<int32_t>(num_candidates);
  p.nfunc = nfunc;
  p.max_seqlen = max_seqlen;
  p.split = l.split;
  p.nsplit = l.nsplit;
  if (func_c && !cand_offsets && l.split < hstu::kPagedMaxSplit) {
    // A mask leaves a CTA less to read than its keys and makes it list its
    // tiles first, so splits are twice as long: one row for each of 128 users
    // under the SLA mask took 25.7 us so and 29.1 us without.
    p.split = std::min(2 * l.split, hstu::kPagedMaxSplit);
    p.nsplit = (max_seqlen + p.split - 1) / p.split;
  }
  p.tensor = l.tensor;
  p.zero = (flags & HSTU_FLAG_ZERO_SKIPPED) != 0;
  p.shorter = l.shorter;
  p.alpha = alpha;
  p.inv_n = 1.0f / static_cast<float>(max_seqlen);
  p.give_up = hstu::handoff_limit() <= 1;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (report && cudaMemsetAsync(ws, 0, hstu::kHdrWords * 4, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  const unsigned blocks = static_cast<unsigned>(static_cast<int64_t>(batch) * p.cache.heads * p.nsplit);
  cudaError_t e;
  if (cache->e4m3) e = half ? hstu::launch_paged_f16_e4m3(p, blocks, cs) : hstu::launch_paged_bf16_e4m3(p, blocks, cs);
  else e = half ? hstu::launch_paged_f16(p, blocks, cs) : hstu::launch_paged_bf16(p, blocks, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"

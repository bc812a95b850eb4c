// Entry points of include/mha_paged.h for the page pool: argument validation and launch on
// the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/mha_paged.h"
#include "buffers.cuh"
#include "common.cuh"
#include "host.cuh"
#include "pages.cuh"

namespace mha {
namespace {

// rows and pages that the kernels step through in 32 bits
constexpr long long kMaxCount = 0x7fffffffLL - (1 << 20);
// entries of a table, and pages that its rows may need: their numbers share a word with
// two bits
constexpr long long kMaxEntries = 0x1fffffffLL;

// page_size: a power of two of at least 16, and tables whose positions fit 32 bits
int check_pages(int num_pages, int page_size, int max_pages, int *shift) {
  if (num_pages < 0 || max_pages < 0) return MHA_ERR_INVALID_ARGUMENT;
  if (page_size <= 0 || (page_size & (page_size - 1)) != 0) return MHA_ERR_INVALID_ARGUMENT;
  if (page_size < 16) return MHA_ERR_UNSUPPORTED;
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  if ((static_cast<long long>(max_pages) << *shift) > (1LL << 31) - 1024) return MHA_ERR_UNSUPPORTED;
  return num_pages <= kMaxCount ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

// A stack of caches: layers x pages x page_size x heads x d.
int check_caches(int layers, int num_pages, int page_size, int H_kv, int d, int layout, int dtype) {
  if (layers < 0 || H_kv < 0 || d <= 0) return MHA_ERR_INVALID_ARGUMENT;
  if (layout != kLayoutBHSD && layout != kLayoutBSHD) return MHA_ERR_INVALID_ARGUMENT;
  if (dtype != MHA_DTYPE_F32 && dtype != MHA_DTYPE_BF16) return MHA_ERR_INVALID_ARGUMENT;
  if (d != 64 && d != 128) return MHA_ERR_UNSUPPORTED;
  return fits({std::max(layers, 1), std::max(num_pages, 1), page_size, H_kv, d})
             ? MHA_OK
             : MHA_ERR_UNSUPPORTED;
}

size_t ints(long long n) { return sizeof(int32_t) * static_cast<size_t>(n); }

}  // namespace
}  // namespace mha

using namespace mha;

extern "C" size_t mha_paged_reserve_workspace_size(int B, int num_pages) {
  if (B < 0 || num_pages < 0 || B > kMaxCount || num_pages > kMaxCount) return 0;
  return round_up(ints(2LL * num_pages + 5LL * B + (num_pages + 31LL) / 32 + kReserveTotals));
}

extern "C" int mha_paged_reserve(const int32_t *block_table, const int32_t *kv_lengths,
                                 const int32_t *new_lengths, const int32_t *parents,
                                 const int32_t *refs, int32_t *table_out, int32_t *lengths_out,
                                 int32_t *refs_out, int32_t *moves, int32_t *counts, int B_old,
                                 int B, int num_pages, int page_size, int max_pages,
                                 void *workspace, size_t workspace_bytes, void *stream) {
  if (B_old < 0 || B < 0) return MHA_ERR_INVALID_ARGUMENT;
  ReserveArgs a{};
  const int st = check_pages(num_pages, page_size, max_pages, &a.page_shift);
  if (st != MHA_OK) return st;
  if (B_old > kMaxCount || B > kMaxCount ||
      static_cast<long long>(B_old) * max_pages > kMaxEntries ||
      static_cast<long long>(B) * (max_pages + 1LL) > kMaxEntries)
    return MHA_ERR_UNSUPPORTED;
  if (B_old == 0 && B == 0 && num_pages == 0 && counts == nullptr) return MHA_OK;
  const size_t nw = mha_paged_reserve_workspace_size(B, num_pages);
  if (workspace_bytes < nw) return MHA_ERR_INVALID_ARGUMENT;
  const Buffer outs[6] = {{refs_out, ints(num_pages), 4},
                          {table_out, ints(static_cast<long long>(B) * max_pages), 4},
                          {lengths_out, ints(B), 4},
                          {moves, ints(2LL * B), 4},
                          {counts, counts != nullptr ? ints(2) : 0, 4},
                          {workspace, nw, kAlign}};
  const Buffer ins[5] = {{refs, ints(num_pages), 4},
                         {block_table, ints(static_cast<long long>(B_old) * max_pages), 4},
                         {kv_lengths, ints(B_old), 4},
                         {new_lengths, ints(B), 4},
                         {parents, parents != nullptr ? ints(B) : 0, 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {0, -1, -1, -1, -1, -1}))
    return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  a.table = block_table;
  a.lens = kv_lengths;
  a.new_lens = new_lengths;
  a.parents = parents;
  a.refs = refs;
  a.table_out = table_out;
  a.lens_out = lengths_out;
  a.refs_out = refs_out;
  a.moves = moves;
  a.counts = counts;
  a.rows = static_cast<int4 *>(workspace);
  a.lowest = reinterpret_cast<int32_t *>(a.rows + B);
  a.given = a.lowest + num_pages;
  a.need = a.given + num_pages;
  a.free = reinterpret_cast<uint32_t *>(a.need + B);
  a.totals = reinterpret_cast<int32_t *>(a.free) + (num_pages + 31LL) / 32;
  a.B_old = B_old;
  a.B = B;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  return launch_reserve(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MHA_OK
                                                                                  : MHA_ERR_CUDA;
}

extern "C" int mha_paged_compact(void *k_cache, void *v_cache, int32_t *lengths_out,
                                 const int32_t *keep, const int32_t *keep_counts,
                                 const int32_t *starts, const int32_t *kv_lengths,
                                 const int32_t *src_table, const int32_t *block_table, int B,
                                 int layers, int H_kv, int d, int num_pages, int page_size,
                                 int max_pages, int max_keep, int layout, int dtype, void *stream) {
  if (B < 0 || max_keep < 0) return MHA_ERR_INVALID_ARGUMENT;
  CompactArgs a{};
  int st = check_pages(num_pages, page_size, max_pages, &a.to.page_shift);
  if (st == MHA_OK) st = check_caches(layers, num_pages, page_size, H_kv, d, layout, dtype);
  if (st != MHA_OK) return st;
  // one CTA to a sequence, head, layer and tensor
  const int heads = std::max(H_kv, 1), stack = std::max(layers, 1);
  // (and a list in 32 bits, with rounds behind it)
  if (max_keep > 1 << 30 || !fits({B, max_pages}) || !fits({B, max_keep}) || !fits({2, B, heads, stack}) ||
      2LL * B * heads * stack > 0x7fffffffLL)
    return MHA_ERR_UNSUPPORTED;
  if (B == 0) return MHA_OK;
  const int row_bytes = d * static_cast<int>(elem_size(dtype));
  const size_t layer =
      static_cast<size_t>(num_pages) * page_size * H_kv * static_cast<size_t>(row_bytes);
  const size_t nc = layer * layers, nt = ints(static_cast<long long>(B) * max_pages);
  const Buffer outs[3] = {{k_cache, nc, 16}, {v_cache, nc, 16}, {lengths_out, ints(B), 4}};
  const Buffer ins[6] = {{keep, ints(static_cast<long long>(B) * max_keep), 4},
                         {keep_counts, ints(B), 4},
                         {starts, starts != nullptr ? ints(B) : 0, 4},
                         {kv_lengths, ints(B), 4},
                         {src_table, src_table != nullptr ? nt : 0, 4},
                         {block_table, nt, 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {-1, -1, -1}))
    return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  a.k = static_cast<uint8_t *>(k_cache);
  a.v = static_cast<uint8_t *>(v_cache);
  a.keep = keep;
  a.counts = keep_counts;
  a.starts = starts;
  a.lens_out = lengths_out;
  a.to.kv_lengths = kv_lengths;
  a.to.block_table = block_table;
  a.to.B = B;
  a.to.num_pages = num_pages;
  a.to.page_size = page_size;
  a.to.max_pages = max_pages;
  a.to.layout = layout;
  a.from = a.to;
  const bool in_place = src_table == nullptr || src_table == block_table;
  if (!in_place) a.from.block_table = src_table;
  a.layer_bytes = static_cast<long long>(layer);
  a.layers = layers;
  a.Hkv = H_kv;
  a.max_keep = max_keep;
  a.row_bytes = row_bytes;
  return launch_compact(a, in_place, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MHA_OK
             : MHA_ERR_CUDA;
}

extern "C" int mha_paged_copy(void *k_cache, void *v_cache, const int32_t *moves, int n, int layers,
                              int H_kv, int d, int num_pages, int page_size, int dtype,
                              void *stream) {
  if (n < 0) return MHA_ERR_INVALID_ARGUMENT;
  int shift = 0;
  int st = check_pages(num_pages, page_size, 0, &shift);
  if (st == MHA_OK) st = check_caches(layers, num_pages, page_size, H_kv, d, kLayoutBHSD, dtype);
  if (st != MHA_OK) return st;
  // pieces of a page in all layers are counted in 32 bits, pairs with a stretch behind them
  const long long page = static_cast<long long>(page_size) * H_kv * d * elem_size(dtype);
  if (n > kMaxCount || !fits({2, layers, page}) || 2LL * layers * (page / 1024 + 1) > 0x7fffffffLL)
    return MHA_ERR_UNSUPPORTED;
  const size_t nc = static_cast<size_t>(page) * num_pages * layers;
  if (n == 0 || nc == 0) return MHA_OK;
  const Buffer outs[2] = {{k_cache, nc, 16}, {v_cache, nc, 16}};
  const Buffer ins[1] = {{moves, ints(2LL * n), 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {-1, -1})) return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  PageCopyArgs a{};
  a.k = static_cast<uint8_t *>(k_cache);
  a.v = static_cast<uint8_t *>(v_cache);
  a.moves = moves;
  a.n = n;
  a.layers = layers;
  a.num_pages = num_pages;
  a.page_bytes = page;
  return launch_page_copy(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MHA_OK
                                                                                    : MHA_ERR_CUDA;
}

// The page pool under the paged cache (include/mha_paged.h): arguments of its kernels, and
// the integer logic that also compiles for the host, where its tests run.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.cuh"

namespace mha {

// ---- tables of the next step (pages_reserve.cu) ------------------------------
struct ReserveArgs {
  const int32_t *table, *lens;  // [B_old, max_pages], [B_old]
  const int32_t *new_lens;      // [B]
  const int32_t *parents;       // [B] or nullptr: row i's is i
  const int32_t *refs;          // [num_pages]
  int32_t *table_out, *lens_out, *refs_out;
  int32_t *moves;   // [B, 2]
  int32_t *counts;  // [2] or nullptr
  // workspace
  int4 *rows;       // [B] what a row keeps: parent, keep, next, last
  int32_t *lowest;  // [num_pages] of a part-filled page: the lowest row that keeps it
  int32_t *given;   // [num_pages] pages given out, in order
  int32_t *need;    // [B] pages that the row needs (kReserve* bits), then its first one's number
  uint32_t *free;   // [num_pages / 32, rounded up] free pages, a bit each
  int32_t *totals;  // [kReserveTotals] pages given out, blocks that are done
  int B_old, B;
  int num_pages, page_shift, max_pages;
};
constexpr int kReserveTotals = 2, kTotalGiven = 0, kTotalDone = 1;
// bits of a row's word beside its number
constexpr int kReserveCopied = 1;  // its part-filled page is replaced by a copy
constexpr int kReserveStays = 2;   // ... stays the row's own
constexpr int kReserveShift = 2;

// What row i of the new tables keeps of its parent, and what it wants.
struct ReserveRow {
  int parent;      // row of the old tables, -1: none
  int keep, next;  // positions kept, and in the end
  int full;        // whole pages kept
  int had, want;   // pages with kept positions, and in the end
  int last;        // the part-filled page among the kept ones; -1: none, or it names no page
};

MHA_HD int reserve_page(const ReserveArgs &a, int row, int idx) {
  const int id = a.table[static_cast<size_t>(row) * a.max_pages + idx];
  return static_cast<unsigned>(id) < static_cast<unsigned>(a.num_pages) ? id : -1;
}
MHA_HD int reserve_clamp(const ReserveArgs &a, int len) {
  const int cap = a.max_pages << a.page_shift;
  return len < 0 ? 0 : (len < cap ? len : cap);
}
MHA_HD int reserve_pages(const ReserveArgs &a, int len) {
  return (len >> a.page_shift) + ((len & ((1 << a.page_shift) - 1)) != 0);
}
MHA_HD ReserveRow reserve_row(const ReserveArgs &a, int i) {
  ReserveRow r;
  r.parent = a.parents != nullptr ? a.parents[i] : i;
  if (static_cast<unsigned>(r.parent) >= static_cast<unsigned>(a.B_old)) r.parent = -1;
  r.next = reserve_clamp(a, a.new_lens[i]);
  const int old = r.parent >= 0 ? reserve_clamp(a, a.lens[r.parent]) : 0;
  r.keep = old < r.next ? old : r.next;
  r.full = r.keep >> a.page_shift;
  r.had = reserve_pages(a, r.keep);
  r.want = reserve_pages(a, r.next);
  r.last = r.had > r.full ? reserve_page(a, r.parent, r.full) : -1;
  return r;
}
// The row's length when it got `got` of the pages that it needs (`copied`: the first was to
// replace its part-filled page).
MHA_HD int reserve_length(const ReserveArgs &a, const ReserveRow &r, bool copied, int got) {
  const int need = r.want - r.had + (copied ? 1 : 0);
  if (got >= need) return r.next;
  if (copied && got <= 0) return r.full << a.page_shift;
  return (r.had + got - (copied ? 1 : 0)) << a.page_shift;
}

cudaError_t launch_reserve(const ReserveArgs &a, int num_sms, cudaStream_t stream);

// ---- tokens that stay, pages that are copied (pages_move.cu) -------------------
struct CompactArgs {
  uint8_t *k, *v;
  const int32_t *keep, *counts, *starts;  // [B, max_keep], [B], [B] or nullptr: zeros
  int32_t *lens_out;
  PagedBatch from, to;  // the tables that positions are read and written by
  long long layer_bytes;
  int layers, Hkv, max_keep;
  int row_bytes;  // of a head
};
// Whether entry i of a list stands, given the one before it (-1: none).
MHA_HD bool compact_stands(int before, int k, int start, int len) {
  return k > before && k < len - start;
}
cudaError_t launch_compact(const CompactArgs &a, bool in_place, int num_sms, cudaStream_t stream);

struct PageCopyArgs {
  uint8_t *k, *v;
  const int32_t *moves;  // [n, 2]
  int n, layers, num_pages;
  long long page_bytes;
};
cudaError_t launch_page_copy(const PageCopyArgs &a, int num_sms, cudaStream_t stream);

// A kernel launch that may begin before the one ahead of it has ended (its griddep_wait
// waits for that), in clusters of `cluster` CTAs.
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, int smem, int cluster,
                          cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace mha

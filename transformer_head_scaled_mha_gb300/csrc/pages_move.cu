// Rows and pages of the paged cache that change places, in all layers at once: the tokens
// of a sequence that stay, moved to the front of their cells or into other pages, and the
// copies of pages that forked sequences may no longer share.
//
// Bound: HBM, twice the moved bytes; for few tokens the chain of loads that finds them
// (count, list, tables, row).  Measured, in captured graphs: the accepted paths (up to 9
// tokens) of 64 trees, 16 layers, 8 heads, d 128: 6.6 us (29 MB moved: 0.65 of a copy's
// rate); 8 sequences of 4096-8192 shortened to three quarters, 4 layers, into other pages:
// 187 us (0.96; 204 with the lists' entries looked at one behind another, 329 with a round's
// places too and one turn of CTAs), in place 214; one such sequence, one layer: 14, in place 26
// (its rounds follow one another);
// 128 pages of 128 KB copied in 16 layers: 165 us (0.96).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pages.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

// Plain loads that the compiler may not move to the read-only path: rows are written by
// this kernel too.
__device__ __forceinline__ uint4 ld16(const uint8_t *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Position and length that sequence b's list counts from and may reach.
struct List {
  int start, len, count;
  const int32_t *keep;
  __device__ __forceinline__ List(const CompactArgs &a, int b) {
    len = max(a.from.kv_lengths[b], 0);
    start = a.starts != nullptr ? min(max(a.starts[b], 0), len) : 0;
    count = min(max(a.counts[b], 0), a.max_keep);
    keep = a.keep + static_cast<size_t>(b) * a.max_keep;
  }
};

// Where an entry's row comes from and goes to, in rows; src < 0: nothing to do.
struct Move {
  long long src, dst;
};
__device__ __forceinline__ Move move_of(const CompactArgs &a, const List &l, int b, int head, int i,
                                        int k) {
  Move m;
  m.src = paged_cell(a.from, b, l.start + k, head, a.Hkv);
  m.dst = paged_cell(a.to, b, l.start + i, head, a.Hkv);
  if (m.dst < 0 || m.src == m.dst) m.src = -1;
  return m;
}

// Lists of up to 32 tokens: a warp per sequence and head, an entry per lane; the rows'
// places are found once for all layers.  A list ascends, so row i comes from place i or
// behind it: rows of a round are all loaded before any is written, and what a later round
// loads lies behind what this one writes.
constexpr int kShort = 32, kShortWarps = 8;
template <int kCols>  // 16-byte columns of a row
__global__ void __launch_bounds__(kShortWarps * 32) compact_short_kernel(const CompactArgs a) {
  constexpr int kRows = 32 / kCols;  // rows side by side in a warp
  constexpr int kDeep = 4;           // ... and behind one another
  __shared__ Move moves[kShortWarps][kShort];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int heads = max(a.Hkv, 1);
  const long long unit = static_cast<long long>(blockIdx.x) * kShortWarps + warp;
  const int b = static_cast<int>(unit / heads), head = static_cast<int>(unit % heads);
  if (b >= a.from.B) return;
  const List l(a, b);
  // (asked for beside the count)
  const int listed = lane < a.max_keep ? l.keep[lane] : -1, k = lane < l.count ? listed : -1;
  const int before = __shfl_up_sync(0xffffffffu, k, 1);
  const unsigned stands = __ballot_sync(
      0xffffffffu, lane < l.count && compact_stands(lane > 0 ? before : -1, k, l.start, l.len));
  const int n = stands == 0xffffffffu ? 32 : __ffs(~stands) - 1;
  if (head == 0 && blockIdx.y == 0 && lane == 0) a.lens_out[b] = l.start + n;
  Move m{-1, -1};
  if (lane < n && a.Hkv > 0) m = move_of(a, l, b, head, lane, k);
  const unsigned moved = __ballot_sync(0xffffffffu, m.src >= 0);
  const int rows = __popc(moved);
  if (m.src >= 0) moves[warp][__popc(moved & ((1u << lane) - 1))] = m;
  __syncwarp();
  const int col = (lane % kCols) * 16, mine = lane / kCols;
  for (int layer = blockIdx.y; layer < a.layers; layer += gridDim.y) {
    const long long base = layer * a.layer_bytes + col;
    for (int r0 = 0; r0 < rows; r0 += kRows * kDeep) {
      uint4 x[2][kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int r = r0 + u * kRows + mine;
        if (r < rows) {
          const long long at = base + moves[warp][r].src * (kCols * 16);
          x[0][u] = ld16(a.k + at);
          x[1][u] = ld16(a.v + at);
        }
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int r = r0 + u * kRows + mine;
        if (r < rows) {
          const long long at = base + moves[warp][r].dst * (kCols * 16);
          st_global_v4(a.k + at, x[0][u]);
          st_global_v4(a.v + at, x[1][u]);
        }
      }
      __syncwarp();
    }
  }
}

// Longer lists: a CTA per sequence, head, layer and tensor (and, where nothing that is
// written is read, stretch of the list), rounds as above.  A round's rows are found while
// those of the round before are on their way.  A CTA may take kPart of a row's kCols columns
// of 16 bytes: its rounds are that much longer, and fewer.
constexpr int kLongThreads = 256, kLongCtas = 4;  // CTAs per SM
template <int kCols, int kPart>
__global__ void __launch_bounds__(kLongThreads, kLongCtas)
    compact_long_kernel(const CompactArgs a, int stretches) {
  constexpr int kRows = kLongThreads / kPart, kDeep = 8, kRound = kRows * kDeep;
  constexpr int kFind = (kRound + kLongThreads - 1) / kLongThreads;  // rows that a thread finds
  static_assert(kCols % kPart == 0, "whole parts");
  // of this round, the next one, and the one before, whose rows may still be on their way out
  __shared__ Move moves[3][kRound];
  __shared__ int stop;
  griddep_launch_dependents();
  griddep_wait();
  const int heads = max(a.Hkv, 1), items = 2 * max(a.layers, 1);
  long long unit = blockIdx.x;
  const int stretch = static_cast<int>(unit % stretches);
  unit /= stretches;
  const int part = static_cast<int>(unit % (kCols / kPart));
  unit /= kCols / kPart;
  const int head = static_cast<int>(unit % heads);
  unit /= heads;
  const int item = static_cast<int>(unit % items), b = static_cast<int>(unit / items);
  const List l(a, b);
  if (threadIdx.x == 0) stop = l.count;
  __syncthreads();
  constexpr int kScan = 8;  // entries in flight
  for (int i0 = threadIdx.x; i0 < l.count; i0 += kScan * kLongThreads) {
    int here[kScan], before[kScan];
#pragma unroll
    for (int s = 0; s < kScan; ++s) {
      const int i = i0 + s * kLongThreads;
      here[s] = i < l.count ? l.keep[i] : 0;
      before[s] = i > 0 && i < l.count ? l.keep[i - 1] : -1;
    }
#pragma unroll
    for (int s = 0; s < kScan; ++s) {
      const int i = i0 + s * kLongThreads;
      if (i < l.count && !compact_stands(before[s], here[s], l.start, l.len)) atomicMin(&stop, i);
    }
  }
  __syncthreads();
  const int n = stop;
  if (head == 0 && item == 0 && stretch == 0 && part == 0 && threadIdx.x == 0) a.lens_out[b] = l.start + n;
  if (a.Hkv == 0 || a.layers == 0) return;
  uint8_t *cache = (item & 1 ? a.v : a.k) + (item >> 1) * a.layer_bytes +
                   (part * kPart + threadIdx.x % kPart) * 16;
  const int mine = threadIdx.x / kPart, step = stretches * kRound;
  // entries of the list that this thread looks up, of the round at r0 (-1: none)
  auto entries = [&](int r0, int (&k)[kFind]) {
#pragma unroll
    for (int f = 0; f < kFind; ++f) {
      const int row = f * kLongThreads + static_cast<int>(threadIdx.x);
      k[f] = row < kRound && r0 + row < n ? l.keep[r0 + row] : -1;
    }
  };
  auto find = [&](Move *to, int r0, const int (&k)[kFind]) {
#pragma unroll
    for (int f = 0; f < kFind; ++f) {
      const int row = f * kLongThreads + static_cast<int>(threadIdx.x);
      if (row >= kRound) break;
      to[row].src = -1;
      if (k[f] >= 0) to[row] = move_of(a, l, b, head, r0 + row, k[f]);
    }
  };
  int r0 = stretch * kRound, k[kFind], buffer = 0;
  entries(r0, k);
  find(moves[0], r0, k);
  entries(r0 + step, k);
  __syncthreads();
  for (; r0 < n; r0 += step) {
    const int behind = buffer == 2 ? 0 : buffer + 1;
    uint4 x[kDeep];
    const Move *m = moves[buffer] + mine;
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (m[u * kRows].src >= 0) x[u] = ld16(cache + m[u * kRows].src * (kCols * 16));
    int next[kFind];
    entries(r0 + 2 * step, next);
    find(moves[behind], r0 + step, k);
#pragma unroll
    for (int f = 0; f < kFind; ++f) k[f] = next[f];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (m[u * kRows].src >= 0) st_global_v4(cache + m[u * kRows].dst * (kCols * 16), x[u]);
    buffer = behind;
  }
}

// Pages: the pairs that name two pages are gathered in shared memory, some at a time, and
// their pages' pieces dealt out to the CTAs.
constexpr int kCopyThreads = 256, kCopyDeep = 4, kPairs = 1024;
constexpr int kPiece = kCopyThreads * kCopyDeep * 16;
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PageCopyArgs a) {
  constexpr int kGroups = kPairs / 32, kWarps = kCopyThreads / 32;
  static_assert(kGroups == 32, "a lane sums over the groups");
  __shared__ int2 pairs[kPairs];
  __shared__ int group[kGroups];  // pairs of each 32
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pieces = static_cast<int>((a.page_bytes + kPiece - 1) / kPiece);
  const long long per_pair = 2LL * a.layers * pieces;
  for (int first = 0; first < a.n; first += kPairs) {
    // (every CTA finds the same order)
    int2 m[kGroups / kWarps];
    unsigned names[kGroups / kWarps];
#pragma unroll
    for (int g = 0; g < kGroups / kWarps; ++g) {
      const int i = first + (g * kWarps + warp) * 32 + lane;
      m[g] = make_int2(-1, -1);
      if (i < a.n)
        m[g] = make_int2(a.moves[2 * static_cast<size_t>(i)], a.moves[2 * static_cast<size_t>(i) + 1]);
      names[g] = __ballot_sync(0xffffffffu,
                               static_cast<unsigned>(m[g].x) < static_cast<unsigned>(a.num_pages) &&
                                   static_cast<unsigned>(m[g].y) < static_cast<unsigned>(a.num_pages) &&
                                   m[g].x != m[g].y);
      if (lane == 0) group[g * kWarps + warp] = __popc(names[g]);
    }
    __syncthreads();
    int sum = group[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const int count = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
    for (int g = 0; g < kGroups / kWarps; ++g) {
      const int at = __shfl_sync(0xffffffffu, sum, g * kWarps + warp) - __popc(names[g]);
      if ((names[g] >> lane) & 1) pairs[at + __popc(names[g] & ((1u << lane) - 1))] = m[g];
    }
    __syncthreads();
    const long long units = count * per_pair;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
      const int2 pair = pairs[u / per_pair];
      const int rest = static_cast<int>(u % per_pair), item = rest / pieces;
      uint8_t *cache = (item & 1) ? a.v : a.k;
      const long long layer = static_cast<long long>(item >> 1) * a.num_pages;
      const long long at = static_cast<long long>(rest % pieces) * kPiece + threadIdx.x * 16;
      const uint8_t *src = cache + (layer + pair.x) * a.page_bytes;
      uint8_t *dst = cache + (layer + pair.y) * a.page_bytes;
      uint4 x[kCopyDeep];
#pragma unroll
      for (int k = 0; k < kCopyDeep; ++k)
        if (at + k * kCopyThreads * 16 < a.page_bytes) x[k] = ld16(src + at + k * kCopyThreads * 16);
#pragma unroll
      for (int k = 0; k < kCopyDeep; ++k)
        if (at + k * kCopyThreads * 16 < a.page_bytes)
          st_global_v4(dst + at + k * kCopyThreads * 16, x[k]);
    }
    __syncthreads();
  }
}

template <int kCols>
cudaError_t compact(const CompactArgs &a, bool in_place, int num_sms, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.from.B) * std::max(a.Hkv, 1);
  if (a.max_keep <= kShort) {
    const long long ctas = (units + kShortWarps - 1) / kShortWarps;
    // layers apart while the SMs have room for more CTAs
    const int apart = static_cast<int>(
        std::max(1LL, std::min<long long>(a.layers, 8LL * num_sms / std::max(ctas, 1LL))));
    return launch_behind(compact_short_kernel<kCols>, dim3(static_cast<unsigned>(ctas), apart),
                         kShortWarps * 32, 0, 1, stream, a);
  }
  const long long all = units * 2 * std::max(a.layers, 1);
  // In place the rounds of a CTA follow one another, and few CTAs leave SMs idle: parts of 64
  // bytes of a row to each while the CTAs all run at once.  One sequence of 8192, 8 heads: d 128
  // bf16 60 -> 29 us, fp32 115 -> 45; 8 of 4096: 54 -> 45; 8 of 4096-8192, 4 layers: 213 -> 219.
  constexpr int kPart = 4;
  if (in_place && all * (kCols / kPart) <= 1LL * kLongCtas * num_sms)
    return launch_behind(compact_long_kernel<kCols, kPart>,
                         dim3(static_cast<unsigned>(all * (kCols / kPart))), kLongThreads, 0, 1,
                         stream, a, 1);
  constexpr int kRound = kLongThreads / kCols * 8;
  const int rounds = (a.max_keep + kRound - 1) / kRound;
  // enough CTAs for several turns of all SMs, so that the last one leaves little idle
  const int stretches = in_place ? 1
                                 : static_cast<int>(std::max(
                                       1LL, std::min<long long>(rounds, 8LL * kLongCtas * num_sms / all)));
  return launch_behind(compact_long_kernel<kCols, kCols>, dim3(static_cast<unsigned>(all * stretches)),
                       kLongThreads, 0, 1, stream, a, stretches);
}

}  // namespace

cudaError_t launch_compact(const CompactArgs &a, bool in_place, int num_sms, cudaStream_t stream) {
  switch (a.row_bytes) {
    case 128: return compact<8>(a, in_place, num_sms, stream);
    case 256: return compact<16>(a, in_place, num_sms, stream);
    case 512: return compact<32>(a, in_place, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_page_copy(const PageCopyArgs &a, int num_sms, cudaStream_t stream) {
  const long long pieces = (a.page_bytes + kPiece - 1) / kPiece;
  const long long units = std::min<long long>(a.n, kPairs) * 2 * a.layers * pieces;
  const int grid = static_cast<int>(std::min<long long>(units, 8LL * num_sms));
  return launch_behind(page_copy_kernel, dim3(std::max(grid, 1)), kCopyThreads, 0, 1, stream, a);
}

}  // namespace mha

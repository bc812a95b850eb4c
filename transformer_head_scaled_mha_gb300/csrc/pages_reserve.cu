// The page tables of the next step: sequences that grow, shrink, fork, end and begin, on
// the device, so that a generation step needs no word from the host.
//
// With old tables and lengths, row i of the new ones keeps the first keep = min(old length
// of its parent, new length) positions of its parent.  Whole pages are shared; a
// part-filled last page will be written, so it has to be the row's own:
//
//   refs'[p] = refs[p] - (old rows' references to p) + (new rows' whole pages that are p)
//   row i keeps its part-filled page p where refs'[p] = 0 and i is the lowest row that
//   keeps p so; then refs'[p] = 1.  Any other such row gets a copy: moves[i] = (p, page).
//   Pages with refs' = 0 are free.  Rows take, in their order, the lowest free ones:
//   the copy first, then those of the positions they grow by; these get refs' = 1.
//
// All of it is integers, and sums that atomics form do not depend on their order.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pages.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kChunk = 256;  // entries of a row that a warp takes at a time

// All threads of the cluster; what they wrote before it is seen behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// refs_out = refs, and the words that the rows' minima start from.
__device__ void begin(const ReserveArgs &a, int thread, int threads) {
  if (a.refs_out != a.refs)
    for (int p = thread; p < a.num_pages; p += threads) a.refs_out[p] = a.refs[p];
  for (int i = thread; i < a.B; i += threads) {
    const ReserveRow r = reserve_row(a, i);
    if (r.last >= 0) a.lowest[r.last] = 0x7fffffff;
  }
}

__device__ __forceinline__ int row_chunks(const ReserveArgs &a) {
  return max(1, (a.max_pages + kChunk - 1) / kChunk);
}

// References given up and taken.  A row that is its own parent keeps its whole pages
// without a word: a step of growing sequences touches none of them.
__device__ void count(const ReserveArgs &a, int warp, int warps) {
  const int lane = threadIdx.x & 31, chunks = row_chunks(a);
  const long long tasks = static_cast<long long>(max(a.B_old, a.B)) * chunks;
  for (long long t = warp; t < tasks; t += warps) {
    const int row = static_cast<int>(t / chunks), from = static_cast<int>(t % chunks) * kChunk;
    int kept = 0;  // whole pages of this row that it keeps itself
    if (row < a.B) {
      const ReserveRow r = reserve_row(a, row);
      if (r.parent == row) {
        kept = r.full;
      } else if (r.parent >= 0) {
        for (int x = from + lane; x < min(r.full, from + kChunk); x += 32) {
          const int p = reserve_page(a, r.parent, x);
          if (p >= 0) atomicAdd(&a.refs_out[p], 1);
        }
      }
      if (from == 0 && lane == 0 && r.last >= 0) atomicMin(&a.lowest[r.last], row);
    }
    if (row < a.B_old) {
      const int had = reserve_pages(a, reserve_clamp(a, a.lens[row]));
      for (int x = max(from, kept) + lane; x < min(had, from + kChunk); x += 32) {
        const int p = reserve_page(a, row, x);
        if (p >= 0) atomicSub(&a.refs_out[p], 1);
      }
    }
  }
}

// Exclusive sum of a number per thread over the block; `total`: of all.
__device__ int block_scan(int x, int *scratch, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int w = scratch[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return inc - x + (warp > 0 ? before : 0);
}

// Which part-filled pages stay, how many pages each row needs, and which free ones it gets.
// One cluster of `ctas`.
__device__ void assign(const ReserveArgs &a, int cta, int ctas) {
  __shared__ int scratch[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // rows: a stretch per CTA, and of it one per thread
  const int per_cta = (a.B + ctas - 1) / ctas, per = (per_cta + kThreads - 1) / kThreads;
  const int stop = min(a.B, (cta + 1) * per_cta);
  const int r0 = min(stop, cta * per_cta + static_cast<int>(threadIdx.x) * per);
  const int r1 = min(stop, r0 + per);
  int mine = 0;
  for (int i = r0; i < r1; ++i) {
    const ReserveRow r = reserve_row(a, i);
    bool copied = false;
    if (r.last >= 0) {
      copied = true;
      // (only the lowest row looks at the page's count, and only it changes it here)
      if (__ldcg(&a.lowest[r.last]) == i) {
        const int refs = __ldcg(&a.refs_out[r.last]);
        if (refs <= 0) {
          __stcg(&a.refs_out[r.last], refs + 1);
          copied = false;
        }
      }
    }
    a.copies[i] = copied;
    a.first[i] = mine;
    mine += r.want - r.had + copied;
  }
  int need, total;
  const int before = block_scan(mine, scratch, need);
  if (threadIdx.x == 0) __stcg(&a.totals[kTotalNeed + cta], need);
  cluster_barrier();
  int at = before;
  total = 0;
  for (int c = 0; c < ctas; ++c) {
    const int n = __ldcg(&a.totals[kTotalNeed + c]);
    if (c < cta) at += n;
    total += n;
  }
  for (int i = r0; i < r1; ++i) a.first[i] += at;
  // free pages: a stretch per warp, whole words of 32
  const int warps = ctas * kWarps;
  const int words = (a.num_pages + 31) / 32, each = (words + warps - 1) / warps;
  const int w0 = min(words, (cta * kWarps + warp) * each), w1 = min(words, w0 + each);
  int found = 0;
#pragma unroll 4
  for (int w = w0; w < w1; ++w) {
    const int p = w * 32 + lane;
    const bool free = p < a.num_pages && __ldcg(&a.refs_out[p]) <= 0;
    found += __popc(__ballot_sync(0xffffffffu, free));
  }
  int of_cta;
  int rank = __shfl_sync(0xffffffffu, block_scan(lane == 0 ? found : 0, scratch, of_cta), 0);
  if (threadIdx.x == 0) __stcg(&a.totals[kTotalFree + cta], of_cta);
  cluster_barrier();
  int all = 0;
  for (int c = 0; c < ctas; ++c) {
    const int n = __ldcg(&a.totals[kTotalFree + c]);
    if (c < cta) rank += n;
    all += n;
  }
  for (int w = w0; w < w1 && rank < total; ++w) {
    const int p = w * 32 + lane;
    const bool free = p < a.num_pages && __ldcg(&a.refs_out[p]) <= 0;
    const unsigned ballot = __ballot_sync(0xffffffffu, free);
    const int to = rank + __popc(ballot & ((1u << lane) - 1));
    if (free && to < total) {
      a.given[to] = p;
      a.refs_out[p] = 1;
    }
    rank += __popc(ballot);
  }
  if (cta == 0 && threadIdx.x == 0) {
    const int given = min(total, all);
    a.totals[kTotalGiven] = given;
    if (a.counts != nullptr) {
      a.counts[0] = given;
      a.counts[1] = all - given;
    }
  }
}

__device__ void write_tables(const ReserveArgs &a, int warp, int warps) {
  const int lane = threadIdx.x & 31, chunks = row_chunks(a);
  const long long tasks = static_cast<long long>(a.B) * chunks;
  const int given = __ldcg(&a.totals[kTotalGiven]);
  for (long long t = warp; t < tasks; t += warps) {
    const int i = static_cast<int>(t / chunks), from = static_cast<int>(t % chunks) * kChunk;
    const ReserveRow r = reserve_row(a, i);
    const int first = __ldcg(&a.first[i]), copied = __ldcg(&a.copies[i]);
    // the k-th of the row's new pages
    auto page = [&](int k) { return first + k < given ? __ldcg(&a.given[first + k]) : -1; };
    int32_t *out = a.table_out + static_cast<size_t>(i) * a.max_pages;
#pragma unroll 4
    for (int x = from + lane; x < min(a.max_pages, from + kChunk); x += 32) {
      int id = -1;
      if (x < r.had && !(copied && x == r.full)) id = reserve_page(a, r.parent, x);
      else if (x < r.want) id = page(x < r.had ? 0 : x - r.had + copied);
      out[x] = id;
    }
    if (from == 0 && lane == 0) {
      const int to = copied ? page(0) : -1;
      a.moves[2 * static_cast<size_t>(i)] = to >= 0 ? r.last : -1;
      a.moves[2 * static_cast<size_t>(i) + 1] = to;
      a.lens_out[i] = reserve_length(a, r, copied != 0, max(given - first, 0));
    }
  }
}

// Everything, one cluster.
__global__ void __launch_bounds__(kThreads) reserve_kernel(const ReserveArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int ctas = gridDim.x, cta = blockIdx.x;
  const int thread = cta * kThreads + threadIdx.x, threads = ctas * kThreads;
  begin(a, thread, threads);
  cluster_barrier();
  count(a, thread >> 5, threads >> 5);
  cluster_barrier();
  assign(a, cta, ctas);
  cluster_barrier();
  write_tables(a, thread >> 5, threads >> 5);
}

// The same in steps over the whole GPU.
__global__ void __launch_bounds__(kThreads) reserve_begin_kernel(const ReserveArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  begin(a, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
}
__global__ void __launch_bounds__(kThreads) reserve_count_kernel(const ReserveArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  count(a, blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps);
}
__global__ void __launch_bounds__(kThreads) reserve_assign_kernel(const ReserveArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  assign(a, blockIdx.x, gridDim.x);
}
__global__ void __launch_bounds__(kThreads) reserve_tables_kernel(const ReserveArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  write_tables(a, blockIdx.x * kWarps + (threadIdx.x >> 5), gridDim.x * kWarps);
}

}  // namespace

cudaError_t launch_reserve(const ReserveArgs &a, int num_sms, cudaStream_t stream) {
  const long long entries = static_cast<long long>(std::max(a.B_old, a.B)) * a.max_pages;
  const int ctas = entries + a.num_pages <= 16384 ? 1 : kReserveMaxCtas;
  if (entries <= 65536)
    return launch_behind(reserve_kernel, dim3(ctas), kThreads, ctas, stream, a);
  const dim3 grid(2 * num_sms);
  cudaError_t e = launch_behind(reserve_begin_kernel, grid, kThreads, 1, stream, a);
  if (e == cudaSuccess) e = launch_behind(reserve_count_kernel, grid, kThreads, 1, stream, a);
  if (e == cudaSuccess) e = launch_behind(reserve_assign_kernel, dim3(ctas), kThreads, ctas, stream, a);
  if (e == cudaSuccess) e = launch_behind(reserve_tables_kernel, grid, kThreads, 1, stream, a);
  return e;
}

}  // namespace mha

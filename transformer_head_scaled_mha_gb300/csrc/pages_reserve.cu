// The page tables of the next step: sequences that grow, shrink, fork, end and begin, on
// the device, so that a generation step needs no word from the host.
//
// With old tables and lengths, row i of the new ones keeps the first keep = min(old length
// of its parent, new length) positions of its parent.  Whole pages are shared; a
// part-filled last page will be written, so it has to be the row's own:
//
//   refs'[p] = refs[p] - (old rows' references to p) + (new rows' whole pages that are p)
//   row i keeps its part-filled page p where refs'[p] <= 0 and i is the lowest row that
//   keeps p so; then refs'[p] grows by one.  Any other such row gets a copy: moves[i] =
//   (p, page).  Pages with refs' <= 0 are free.  Rows take, in their order, the lowest free
//   ones: the copy first, then those of the positions they grow by; these get refs' = 1.
//
// All of it is integers, and sums and minima that atomics form do not depend on their
// order.  A row that is its own parent keeps its whole pages without a word, so that a step
// of growing sequences counts almost nothing, and a page that a beam shared with its parent
// is given up and taken without one.
//
// Bound: the way from number to number (parents, lengths, tables, counts, ranks, pages), not
// the few bytes.  Measured, in captured graphs: 256 sequences of 128-1024 positions, pages of
// 16, one step: 8.9 us, with tables for 8192 and more 11.1 to 11.6 (15.2 as one cluster with the
// counts in L2, 13.2 as one block that writes all tables); 8 of 300: 5.5; 64 beams of 2000-8000,
// 459 pages to a row: 14.1; 1024 beams of 2048-8192, 513 pages to a row, 350000 pages: 19 (54.7
// as one cluster of 8 CTAs, 34.6 of 16; 20.2 in blocks of 1024, which leave the next launch no
// room; a fifth launch in place of the last block: 1.3 less, but 2 more of the host's time).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pages.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kChunk = 256;  // entries of a row that a warp takes at a time

__device__ __forceinline__ int row_chunks(const ReserveArgs &a) {
  return max(1, (a.max_pages + kChunk - 1) / kChunk);
}

// A row in 16 bytes: what took loads behind one another to find.
__device__ __forceinline__ int4 pack(const ReserveRow &r) {
  return make_int4(r.parent, r.keep, r.next, r.last);
}
__device__ __forceinline__ ReserveRow unpack(const ReserveArgs &a, int4 s) {
  ReserveRow r;
  r.parent = s.x;
  r.keep = s.y;
  r.next = s.z;
  r.last = s.w;
  r.full = r.keep >> a.page_shift;
  r.had = reserve_pages(a, r.keep);
  r.want = reserve_pages(a, r.next);
  return r;
}

// An entry that names no page is -1.
__device__ __forceinline__ int named(const ReserveArgs &a, int id) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(a.num_pages) ? id : -1;
}

// References given up and taken in entries [from, from + kChunk) of old and new row `row`,
// added to `refs`; by a warp.  A page that the row had at that place and keeps there (its
// own, or one it shared with its parent) is given up and taken: no word.  `had`: pages of
// the old row.
__device__ __forceinline__ void count_chunk(const ReserveArgs &a, int row, const ReserveRow &r, int had,
                                            int from, int *refs) {
  const int lane = threadIdx.x & 31;
  const bool same = r.parent == row;  // whole pages that the row keeps itself: none to look at
  const int32_t *mine = a.table + static_cast<size_t>(row) * a.max_pages;
  const int32_t *parents = a.table + static_cast<size_t>(max(r.parent, 0)) * a.max_pages;
  constexpr int kDeep = 4;
  for (int x0 = from + lane; x0 < min(max(had, r.full), from + kChunk); x0 += 32 * kDeep) {
    int old[kDeep], now[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int x = x0 + 32 * k;
      const bool in = x < from + kChunk;
      old[k] = now[k] = -1;
      if (in && x < had && !(same && x < r.full)) old[k] = __ldcg(mine + x);
      if (in && x < r.full && !same) now[k] = __ldcg(parents + x);
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      if (old[k] == now[k]) continue;
      const int gone = named(a, old[k]), taken = named(a, now[k]);
      if (gone >= 0) atomicSub(&refs[gone], 1);
      if (taken >= 0) atomicAdd(&refs[taken], 1);
    }
  }
}

// What row i needs: pages, and whether its part-filled page, with its references and the
// lowest row that keeps it, stays or is copied.
__device__ __forceinline__ int need_of(const ReserveRow &r, int i, int lowest, int refs) {
  int bits = 0;
  if (r.last >= 0) bits = lowest == i && refs <= 0 ? kReserveStays : kReserveCopied;
  return (r.want - r.had + ((bits & kReserveCopied) != 0)) << kReserveShift | bits;
}

// Exclusive sum of a number per thread over a block of kT; `total`: of all.
template <int kT>
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
  int w = lane < kT / 32 ? scratch[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return inc - x + (warp > 0 ? before : 0);
}

// Gives out the `total` lowest free pages, whose bits `free` tells by words, to `given`; refs[p] =
// 1.  One block: runs of 32 words are counted by the warps in turn, summed, and those that
// hold pages to give looked at again.  Returns how many there were to give; `all`: how many
// were free.
template <int kT, typename Page, typename Free>
__device__ int give_pages(const ReserveArgs &a, const Free &free, int total, int *refs,
                          Page *given, int *scratch, int *runs, int &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = (a.num_pages + 31) / 32;
  all = 0;  // so far
  for (int base = 0; base < words; base += 32 * kT) {
    __syncthreads();
    constexpr int kDeep = 8;
    for (int s = warp; s < kT && base + s * 32 < words; s += kDeep * (kT / 32)) {
      uint32_t bits[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int w = base + (s + k * (kT / 32)) * 32 + lane;
        bits[k] = s + k * (kT / 32) < kT && w < words ? free(w) : 0u;
      }
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int n = __reduce_add_sync(0xffffffffu, __popc(bits[k]));
        if (lane == 0 && s + k * (kT / 32) < kT) runs[s + k * (kT / 32)] = n;
      }
    }
    __syncthreads();
    int sum;
    const bool is = base + static_cast<int>(threadIdx.x) * 32 < words;
    const int before = all + block_scan<kT>(is ? runs[threadIdx.x] : 0, scratch, sum);
    runs[threadIdx.x] = before;
    all += sum;
    __syncthreads();
    for (int s = warp; s < kT && base + s * 32 < words && runs[s] < total; s += (kT / 32)) {
      const int w = base + s * 32 + lane;
      uint32_t bits = w < words ? free(w) : 0u;
      int inc = __popc(bits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      for (int to = runs[s] + inc - __popc(bits); bits != 0 && to < total; bits &= bits - 1, ++to) {
        const int p = w * 32 + __ffs(bits) - 1;
        given[to] = static_cast<Page>(p);
        refs[p] = 1;
      }
    }
  }
  return min(total, all);
}
__device__ __forceinline__ void write_counts(const ReserveArgs &a, int given, int all) {
  if (a.counts == nullptr) return;
  a.counts[0] = given;
  a.counts[1] = all - given;
}

// Where a new row's entries come from: those before `end` from its parent's row, at `from`;
// entry x from there to `want` is the (shift + x)-th of the pages given out.
struct Source {
  int from, end, want, shift;
};
__device__ __forceinline__ Source source_of(const ReserveArgs &a, const ReserveRow &r, int word) {
  Source s;
  s.from = max(r.parent, 0) * a.max_pages;
  s.end = word & kReserveCopied ? r.full : r.had;
  s.want = r.want;
  s.shift = (word >> kReserveShift) - s.end;
  return s;
}
// Entry x, a number of the parent's row as it is: loads that nothing looks at yet go out
// one behind another.
template <typename Page>
__device__ __forceinline__ int entry(const ReserveArgs &a, const Source &s, int x, const Page *given,
                                     int count) {
  int id = -1;
  if (x < s.end) id = __ldcg(a.table + s.from + x);
  if (x >= s.end && x < s.want && s.shift + x < count) id = given[s.shift + x];
  return id;
}

// A new row's other results; by one thread.
template <typename Page>
__device__ __forceinline__ void write_row(const ReserveArgs &a, int i, const ReserveRow &r, int word,
                                          const Page *given, int count) {
  const int first = word >> kReserveShift;
  const bool copied = (word & kReserveCopied) != 0;
  const int to = copied && first < count ? static_cast<int>(given[first]) : -1;
  a.moves[2 * static_cast<size_t>(i)] = to >= 0 ? r.last : -1;
  a.moves[2 * static_cast<size_t>(i) + 1] = to;
  a.lens_out[i] = reserve_length(a, r, copied, max(count - first, 0));
}

// ---- one cluster -----------------------------------------------------------------
// For pools and tables that one SM goes through in a moment: the references, the rows and
// the pages given out live in shared memory, and barriers of a block stand between the
// steps.  Every CTA of the cluster does all of it alike, in its own shared memory, and
// writes a share of the results: copying the tables is most of the work, and that much
// faster than telling the others.
//
// Rows and pages by what fits shared memory; entries, with the rows' empty places, by the time
// that they take.  Measured, one cluster / the whole GPU: one step of 256 sequences of 128-1024,
// pages of 16, room for 2048: 9.1 / 11.1 us, 4096 (65536 entries): 9.7 / 11.0, 8192: 12.0 / 11.3,
// 32768: 23.9 / 11.6; of 64: 65536 entries 8.8 / 10.8, 131072 10.6 / 10.6, 262144 14.5 / 10.6; of
// 1024 of 100-400: 65536 13.9 / 14.1, 131072 15.6 / 13.8.  Beams, which count all their pages,
// would go to the whole GPU earlier: 64 of 2000-4000, 32768 entries: 13.6 / 11.6, 65536 18.0 /
// 11.7; 32 of 1000-8000, 16384: 9.9 / 11.1, 32768 12.2 / 10.7.
constexpr int kSmallRows = 1024, kSmallPages = 28672;
constexpr int kSmallEntries = 65536;  // of the tables
constexpr int kSmallCtas = 8;
constexpr int kFew = 4;  // references that a thread counts alone
struct SmallShared {
  int4 rows[kSmallRows];
  Source sources[kSmallRows];
  int had[kSmallRows], listed[kSmallRows], count;
  int runs[kThreads];
  uint32_t free[kSmallPages / 32];
  int scratch[kWarps];
  uint16_t given[kSmallPages];  // before: of a part-filled page, the lowest row that keeps it
  int refs[kSmallPages];        // (only num_pages of them are there)
};
static_assert(kSmallRows < 0xffff && kSmallPages <= 0x10000 && sizeof(SmallShared) <= 232448, "sizes");

// at[i] = min(at[i], x), others' at[i ^ 1] untouched
__device__ __forceinline__ void atomic_min16(uint16_t *at, int i, uint32_t x) {
  uint32_t *word = reinterpret_cast<uint32_t *>(at + (i & ~1));
  const int shift = (i & 1) * 16;
  uint32_t old = *reinterpret_cast<volatile uint32_t *>(word);
  while (((old >> shift) & 0xffffu) > x) {
    const uint32_t seen = old;
    old = atomicCAS(word, seen, (seen & ~(0xffffu << shift)) | x << shift);
    if (old == seen) break;
  }
}

__global__ void __launch_bounds__(kThreads) reserve_small_kernel(const ReserveArgs a) {
  const int cta = blockIdx.x, ctas = gridDim.x;
  extern __shared__ __align__(16) uint8_t smem[];
  SmallShared &sh = *reinterpret_cast<SmallShared *>(smem);
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = row_chunks(a);
  const int mine = threadIdx.x;  // this thread's row
#pragma unroll 8
  for (int p = threadIdx.x; p < a.num_pages; p += kThreads) sh.refs[p] = a.refs[p];
  ReserveRow r{};
  r.parent = r.last = -1;
  // pages of the old row of that number
  const int had = mine < a.B_old ? reserve_pages(a, reserve_clamp(a, a.lens[mine])) : 0;
  if (threadIdx.x == 0) sh.count = 0;
  sh.had[mine] = had;
  if (mine < a.B) r = reserve_row(a, mine);
  sh.rows[mine] = pack(r);
  if (mine < a.B) {
    if (r.last >= 0) sh.given[r.last] = 0xffff;
  }
  __syncthreads();
  // every CTA has read refs, which refs_out may be (waited for below)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (r.last >= 0) atomic_min16(sh.given, r.last, mine);
  // rows with few references to count, one to a thread; the others by warps
  const int kept = r.parent == mine ? r.full : 0;  // whole pages that the row keeps itself
  if (max(had - kept, 0) + (r.parent != mine ? r.full : 0) <= kFew) {
    for (int x = kept; x < had; ++x) {
      const int p = reserve_page(a, mine, x);
      if (p >= 0) atomicSub(&sh.refs[p], 1);
    }
    for (int x = 0; r.parent != mine && x < r.full; ++x) {
      const int p = reserve_page(a, r.parent, x);
      if (p >= 0) atomicAdd(&sh.refs[p], 1);
    }
  } else {
    sh.listed[atomicAdd(&sh.count, 1)] = mine;  // (in any order: sums)
  }
  __syncthreads();
  for (int t = warp; t < sh.count * chunks; t += kWarps) {
    const int row = sh.listed[t / chunks];
    count_chunk(a, row, unpack(a, sh.rows[row]), sh.had[row], t % chunks * kChunk, sh.refs);
  }
  __syncthreads();
  int word = 0, total, given;
  if (mine < a.B)
    word = r.last >= 0 ? need_of(r, mine, sh.given[r.last], sh.refs[r.last]) : need_of(r, mine, -1, 0);
  const int before = block_scan<kThreads>(word >> kReserveShift, sh.scratch, total);
  word = before << kReserveShift | (word & ((1 << kReserveShift) - 1));
  sh.sources[mine] = source_of(a, r, word);
  // (every row has looked at its page's references: the scan's barriers)
  if (word & kReserveStays) ++sh.refs[r.last];
  __syncthreads();
  for (int w = warp; w < (a.num_pages + 31) / 32; w += kWarps) {
    const int p = w * 32 + lane;
    const unsigned free = __ballot_sync(0xffffffffu, p < a.num_pages && sh.refs[p] <= 0);
    if (lane == 0) sh.free[w] = free;
  }
  __syncthreads();
  int all;
  given = give_pages<kThreads>(a, [&](int w) { return sh.free[w]; }, total, sh.refs, sh.given, sh.scratch, sh.runs, all);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  for (int p = cta * kThreads + threadIdx.x; p < a.num_pages; p += ctas * kThreads)
    a.refs_out[p] = sh.refs[p];
  if (mine < a.B && mine % ctas == cta) write_row(a, mine, r, word, sh.given, given);
  if (cta == 0 && threadIdx.x == 0) write_counts(a, given, all);
  // the entries of all rows behind one another, some loads in flight to a thread
  constexpr int kDeep = 8;
  const int width = max(a.max_pages, 1), entries = a.B * a.max_pages, step = ctas * kThreads;
  const int rows_on = step / width, cols_on = step % width;
  const int first = cta * kThreads + threadIdx.x;
  int row = first / width, x = first % width;
  for (int e = first; e < entries; e += kDeep * step) {
    int id[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      id[k] = e + k * step < entries ? entry(a, sh.sources[row], x, sh.given, given) : -1;
      row += rows_on;
      x += cols_on;
      if (x >= width) {
        x -= width;
        ++row;
      }
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (e + k * step < entries) a.table_out[e + k * step] = named(a, id[k]);
  }
}

// ---- larger ones: the whole GPU, a launch to a step -----------------------------------
// (__ldcg: numbers that other SMs have just written, or the launch ahead, which may still run
// when this one begins.)  Blocks of 512 leave room on an SM for the next launch's, which then
// wait there.
constexpr int kStepThreads = 512, kStepWarps = kStepThreads / 32;

__device__ void begin_step(const ReserveArgs &a, int block, int blocks) {
  const int thread = block * kStepThreads + threadIdx.x, threads = blocks * kStepThreads;
  if (a.refs_out != a.refs) {
#pragma unroll 4
    for (int p = thread; p < a.num_pages; p += threads) a.refs_out[p] = __ldcg(a.refs + p);
  }
  if (thread == 0) a.totals[kTotalDone] = 0;
  for (int i = thread; i < a.B; i += threads) {
    const ReserveRow r = reserve_row(a, i);
    a.rows[i] = pack(r);
    if (r.last >= 0) a.lowest[r.last] = 0x7fffffff;
  }
}

__device__ void count_step(const ReserveArgs &a, int block, int blocks) {
  const int chunks = row_chunks(a), warps = blocks * kStepWarps;
  const long long tasks = static_cast<long long>(max(a.B_old, a.B)) * chunks;
  for (long long t = block * kStepWarps + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int row = static_cast<int>(t / chunks), from = static_cast<int>(t % chunks) * kChunk;
    ReserveRow r{};
    r.parent = r.last = -1;
    if (row < a.B) r = unpack(a, __ldcg(&a.rows[row]));
    const int had = row < a.B_old ? reserve_pages(a, reserve_clamp(a, a.lens[row])) : 0;
    count_chunk(a, row, r, had, from, a.refs_out);
    if (from == 0 && (threadIdx.x & 31) == 0 && r.last >= 0) atomicMin(&a.lowest[r.last], row);
  }
}

// Pages that stay, the rows' first numbers, and the pages given out: by one block.
__device__ void give_step(const ReserveArgs &a) {
  __shared__ int scratch[kStepWarps], runs[kStepThreads];
  int total = 0;
  for (int base = 0; base < a.B; base += kStepThreads) {
    const int i = base + threadIdx.x;
    const int word = i < a.B ? __ldcg(&a.need[i]) : 0;
    const int last = i < a.B ? __ldcg(&a.rows[i].w) : 0;
    int refs = -1;  // (one row to a page)
    if (word & kReserveStays) refs = atomicAdd(&a.refs_out[last], 1);
    int sum;
    const int before = total + block_scan<kStepThreads>(word >> kReserveShift, scratch, sum);
    if (i < a.B) a.need[i] = before << kReserveShift | (word & ((1 << kReserveShift) - 1));
    // (a page whose references were fewer than the old rows that held it stays free)
    if (refs == 0) atomicAnd(&a.free[last >> 5], ~(1u << (last & 31)));
    total += sum;
  }
  __syncthreads();
  int all;
  const int given = give_pages<kStepThreads>(a, [&](int w) { return __ldcg(&a.free[w]); }, total, a.refs_out, a.given, scratch, runs, all);
  if (threadIdx.x == 0) {
    a.totals[kTotalGiven] = given;
    write_counts(a, given, all);
  }
}

// What rows need, and which pages are free but for those that stay; the block that is done
// last gives them out.
__device__ void need_step(const ReserveArgs &a, int block, int blocks) {
  const int thread = block * kStepThreads + threadIdx.x, threads = blocks * kStepThreads;
  for (int i = thread; i < a.B; i += threads) {
    const ReserveRow r = unpack(a, __ldcg(&a.rows[i]));
    a.need[i] = r.last >= 0 ? need_of(r, i, __ldcg(&a.lowest[r.last]), __ldcg(&a.refs_out[r.last]))
                            : need_of(r, i, -1, 0);
  }
  const int words = (a.num_pages + 31) / 32, lane = threadIdx.x & 31;
#pragma unroll 4
  for (int w = thread >> 5; w < words; w += threads >> 5) {
    const int p = w * 32 + lane;
    const unsigned free = __ballot_sync(0xffffffffu, p < a.num_pages && __ldcg(&a.refs_out[p]) <= 0);
    if (lane == 0) a.free[w] = free;
  }
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(&a.totals[kTotalDone], 1) == blocks - 1;
  }
  __syncthreads();
  if (last) {
    __threadfence();
    give_step(a);
  }
}

__device__ void tables_step(const ReserveArgs &a, int block, int blocks) {
  const int chunks = row_chunks(a), warps = blocks * kStepWarps, given = __ldcg(&a.totals[kTotalGiven]);
  const int lane = threadIdx.x & 31;
  const long long tasks = static_cast<long long>(a.B) * chunks;
  for (long long t = block * kStepWarps + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int i = static_cast<int>(t / chunks), from = static_cast<int>(t % chunks) * kChunk;
    const ReserveRow r = unpack(a, __ldcg(&a.rows[i]));
    const int word = __ldcg(&a.need[i]);
    const Source src = source_of(a, r, word);
    int id[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) id[k] = entry(a, src, from + lane + 32 * k, a.given, given);
    int32_t *out = a.table_out + static_cast<size_t>(i) * a.max_pages + from + lane;
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k)
      if (from + lane + 32 * k < a.max_pages) out[32 * k] = named(a, id[k]);
    if (from == 0 && lane == 0) write_row(a, i, r, word, a.given, given);
  }
}

// The whole GPU, a launch to a step.
template <void (*kStep)(const ReserveArgs &, int, int)>
__global__ void __launch_bounds__(kStepThreads) reserve_step_kernel(const ReserveArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  kStep(a, blockIdx.x, gridDim.x);
}

}  // namespace

cudaError_t launch_reserve(const ReserveArgs &a, int num_sms, cudaStream_t stream) {
  const long long entries = static_cast<long long>(std::max(a.B_old, a.B)) * a.max_pages;
  if (std::max(a.B_old, a.B) <= kSmallRows && a.num_pages <= kSmallPages && entries <= kSmallEntries) {
    const int smem = static_cast<int>(sizeof(SmallShared) - sizeof(int) * kSmallPages) + 4 * a.num_pages;
    const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(reserve_small_kernel),
                                        static_cast<int>(sizeof(SmallShared)));
    if (e != cudaSuccess) return e;
    // two entries to a thread
    const int ctas = static_cast<int>(std::min<long long>(kSmallCtas, 1 + entries / (2 * kThreads)));
    return launch_behind(reserve_small_kernel, dim3(ctas), kThreads, smem, ctas, stream, a);
  }
  const dim3 grid(2 * num_sms);
  cudaError_t e = launch_behind(reserve_step_kernel<begin_step>, grid, kStepThreads, 0, 1, stream, a);
  if (e == cudaSuccess)
    e = launch_behind(reserve_step_kernel<count_step>, grid, kStepThreads, 0, 1, stream, a);
  if (e == cudaSuccess)
    e = launch_behind(reserve_step_kernel<need_step>, grid, kStepThreads, 0, 1, stream, a);
  if (e == cudaSuccess)
    e = launch_behind(reserve_step_kernel<tables_step>, grid, kStepThreads, 0, 1, stream, a);
  return e;
}

}  // namespace mha

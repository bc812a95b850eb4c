// Attention over a paged fp32 key/value cache on the CUDA cores (FFMA, no TF32), and
// the joining of split units that every paged attention kernel uses.
//
// A CTA of four warps walks its parts (paged.cuh): R <= 16 query rows of one
// key/value head against tiles of 128 keys (large trees at d 128: 32 rows, the second
// 16 by four warps of their own).  Warp w takes keys 32 w .. 32 w + 31
// of each tile: scores with up to 4 keys and 4 rows to a lane (keys staged in shared memory,
// rows padded by 16 bytes so that lanes read without conflicts), an online
// softmax with a row per lane, or 32 / R lanes to a row, through a small square of
// shared memory, then the value rows, up to 8 rows and d / 16 output columns to a lane.  Keys and
// values are copied to shared memory without registers (cp.async): the next tile's keys
// while this one's softmax and values are worked on, its values while the next scores
// are, so a warp always has a tile in flight.  The warps' sums are joined once per part.
//
// Bound: few parts per CTA, so the time from launch to the first score and the code's
// own way into the instruction caches; hence one copy loop for both ends of a tile
// (the walk starts one tile early, with nothing to work on) and rows' places and
// limits in shared memory, found once.  Measured, with the merge: 8 sequences of 90-700
// keys, 5 tokens of 8 heads over 2, d 64: 17.0 us (44 with two tiles to a CTA and rows in
// registers); one token, 16 sequences of 1000-4000 keys, 32 heads over 8, d 128: 62 us,
// 5.4 TB/s; 4 tokens, 8 such sequences: 61 us, 2.7 TB/s.  Chunks and prompts take it as
// well, 16 rows at a time, each of which reads the keys again: 4 x 2048 tokens of 16 heads,
// d 64: 1111 us, 31 TFLOP/s (1383 with one key and all rows to a lane in the scores and one
// row of all in the output: a wide load takes 4 cycles to its registers even where all lanes
// ask for the same); d 128: 2610 us, 26 TFLOP/s (0.3 of the CUDA cores' nominal
// 80); 16 trees of 32 drafted tokens over 1000-2000 keys, 16 heads, d 64: 120 us, 25
// TFLOP/s.  Bound there by latencies between two warps to a scheduler (at d 128 one), which
// shared memory has no room to add to: 0.45 to 0.59 of the issue slots, 0.5 to 0.65 of the
// loads' wavefronts.  Hence units of 32 rows for larger trees at d 128, whose second 16 have
// four warps of their own over the same keys: 16 trees of 150 tokens of 12 heads over 4, 300
// keys: 282 us, 211 so (d 64, where the registers no longer suffice: 122, 116, and smaller
// ones slower).  Trees come in units of 4 or 8 rows where there is little work: 8 of 5-13
// tokens over 90-700 keys, 8 heads over 2, d 64: 15 us (19); and of up to 8 where a tree has
// no more: 16 of 8 tokens of 8 heads over 6000 keys, d 64: 80 us (105 as 16 rows).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kRows = 16;
constexpr int kKeys = 32;  // keys of a warp per tile

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// a lane's 2 or 4 columns of a row of sums, and of a row of output
__device__ __forceinline__ void ld_cols(const float *p, float (&x)[2]) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  x[0] = v.x;
  x[1] = v.y;
}
__device__ __forceinline__ void ld_cols(const float *p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x;
  x[1] = v.y;
  x[2] = v.z;
  x[3] = v.w;
}
__device__ __forceinline__ void st_cols(float *p, const float (&x)[2]) {
  *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}
__device__ __forceinline__ void st_cols(float *p, const float (&x)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void st_cols(__nv_bfloat16 *p, const float (&x)[2]) {
  *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(x[0], x[1]);
}
__device__ __forceinline__ void st_cols(__nv_bfloat16 *p, const float (&x)[4]) {
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// 16 bytes global -> shared, or zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t saddr, const void *gptr, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(saddr), "l"(gptr),
               "r"(there ? 16 : 0)
               : "memory");
}
// all but the last N groups of this thread's copies are complete
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// N floats, as wide as they come
template <int N>
__device__ __forceinline__ void ld_vec(const float *p, float *x) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(p + i);
      x[i] = v.x;
      x[i + 1] = v.y;
      x[i + 2] = v.z;
      x[i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2 *>(p);
    x[0] = v.x;
    x[1] = v.y;
  } else {
    static_assert(N == 1, "widths");
    x[0] = *p;
  }
}
template <int N>
__device__ __forceinline__ void st_vec(float *p, const float *x) {
  if constexpr (N == 4) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else if constexpr (N == 2) {
    *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
  } else {
    static_assert(N == 1, "widths");
    *p = x[0];
  }
}

template <int D, int kSets>
struct Smem {
  float q[kSets * kRows][D];
  float k[kWarps][kKeys][D + 4];
  float v[kWarps][kKeys][D];                  // at a part's end the warps' sums
  float p[kSets * kWarps][kKeys][kRows + 4];  // scores, then their powers
  float alpha[kSets * kWarps][kRows];         // what the older sums shrink to
  float m[kSets * kWarps][kRows], l[kSets * kWarps][kRows];
  float f[kSets * kWarps][kRows], total[kSets * kRows];  // the warps' weights when joined, the sum
  long long row[kSets * kRows];  // where a row's query and output begin (-1: no row)
  int lim[kSets * kRows];        // keys below this are allowed (of a tree: the row's token, -1:
                                 // no row)
  long long scratch[40];
};

// kSets: of RP rows, each with four warps of its own over the same keys and values.
template <int D, int RP, bool kTree, int kSets>
__global__ void __launch_bounds__(kSets * kThreads, kSets == 1 ? 2 : 1)
    paged_simt_kernel(const __grid_constant__ PagedProblem p) {
  // A lane's squares: scores of kTR rows and kTK keys (kKg apart), output of kOR rows and kOC
  // columns (pieces of kOV, kOg lanes side by side).
  constexpr int kTR = RP == 16 ? 4 : (RP == 1 ? 1 : 2), kTK = RP / kTR, kKg = 32 / kTK;
  constexpr int kOR = RP <= 4 ? RP : RP / 2, kOC = RP * D / 32 / kOR, kOV = kOC < 4 ? kOC : 4;
  constexpr int kOg = D / kOC;
  constexpr int kPer = 32 / RP;  // lanes to a row in the softmax
  constexpr int kAll = kSets * RP;  // rows of a unit
  static_assert(kSets * kRows <= kKeys && (kSets == 1 || RP == kRows),
                "the warps' sums fit where their values were");
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D, kSets> &sm = *reinterpret_cast<Smem<D, kSets> *>(smem_raw);
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = warp % kWarps, set = warp / kWarps;  // whose keys, whose rows
  const PagedSpan span = paged_span<kSets * kThreads>(p, blockIdx.x, gridDim.x, sm.scratch);
  PagedWalk walk;
  walk.begin(p, span);
  PagedPart part;
  int flags = 0, mrow = 0, mtokens = 0, mhead = 0, mheads = 0;
  const float *q = static_cast<const float *>(p.q);
  const float *kc = static_cast<const float *>(p.k), *vc = static_cast<const float *>(p.v);
  float *out = static_cast<float *>(p.out);
  float *kw = &sm.k[slice][0][0], *vw = &sm.v[slice][0][0];
  const int key_at = lane % kKg, row_at = lane / kKg * kTR;           // of its scores
  const int col_at = lane % kOg * kOV, orow_at = lane / kOg * kOR;  // of its output
  // the warps of a slice wait for one another
  auto slice_sync = [&]() {
    if constexpr (kSets == 1) {
      __syncwarp();
    } else {
      asm volatile("bar.sync %0, %1;" ::"r"(1 + slice), "n"(kSets * 32) : "memory");
    }
  };
  // copies the slice's 32 cache rows, one per lane's cell, zeros where there is none; 16
  // bytes per lane, a share of the rows to each of its warps
  auto copy = [&](const float *cache, float *to, int stride, long long cell) {
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;  // lanes per row, rows at once
    const int c = (lane % kLanes) * 4;
#pragma unroll 4
    for (int j = 0; j < kKeys / kSets; j += kAtOnce) {
      const int row = set * (kKeys / kSets) + j + lane / kLanes;
      const long long at = __shfl_sync(0xffffffffu, cell, row);
      cp_async16_or_zero(smem_addr(to + row * stride + c), cache + (at < 0 ? 0 : at) * D + c,
                         at >= 0);
    }
    cp_async_commit();
  };
  while (walk.next(p, part)) {
    __syncthreads();  // the part before has read q and the warps' sums
    if (threadIdx.x < kAll) {
      const int r = threadIdx.x, h = r / p.tb, i = part.i0 + r - h * p.tb;
      sm.row[r] = h < part.heads && i < part.i1
                      ? (static_cast<long long>(part.seq.q0 + i) * p.H + part.h0 + h) * D
                      : -1;
      // of a tree: the row's token
      sm.lim[r] = kTree ? (h < part.heads && i < part.i1 ? part.seq.q0 + i : -1)
                        : paged_kv_end(part.seq, i + 1, p.causal);
    }
    __syncthreads();
    for (int e = threadIdx.x * 4; e < kAll * D; e += kSets * kThreads * 4) {
      const long long row = sm.row[e / D];
      *reinterpret_cast<float4 *>(&sm.q[0][e]) =
          row >= 0 ? *reinterpret_cast<const float4 *>(q + row + e % D) : make_float4(0, 0, 0, 0);
    }
    const int mine = lane % RP, lim = sm.lim[set * RP + mine];  // this lane's row in the softmax
    const uint32_t *tree = kTree && lim >= 0 ? p.tree + static_cast<size_t>(lim) * p.tree_words : nullptr;
    float m = -INFINITY, l = 0.f;                    // ... its maximum, and its share of the sum
    float acc[kOR][kOC];
#pragma unroll
    for (int r = 0; r < kOR; ++r)
#pragma unroll
      for (int c = 0; c < kOC; ++c) acc[r][c] = 0.f;
    __syncthreads();
    long long cell = -1;
#pragma unroll 1
    for (int t = part.t0 - 1; t < part.t1; ++t) {
      const bool work = t >= part.t0;
      const int first = t * kPagedTile + slice * kKeys;  // this warp's keys
      // the next tile's cache row, one per lane (-1: none)
      const int ahead = first + kPagedTile + lane;
      const long long next = t + 1 < part.t1 && ahead < part.kv_end
                                 ? paged_cell(p.batch, part.b, ahead, part.kv, p.Hkv)
                                 : -1;
      if (work) {
        cp_async_wait<1>();  // this tile's keys (its values may be on their way)
        slice_sync();
        float s[kTK][kTR];
#pragma unroll
        for (int x = 0; x < kTK; ++x)
#pragma unroll
          for (int r = 0; r < kTR; ++r) s[x][r] = 0.f;
#pragma unroll 8
        for (int c = 0; c < D; c += 4) {
          float4 kv[kTK];
#pragma unroll
          for (int x = 0; x < kTK; ++x)
            kv[x] = *reinterpret_cast<const float4 *>(&sm.k[slice][key_at + x * kKg][c]);
#pragma unroll
          for (int r = 0; r < kTR; ++r) {
            const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[set * RP + row_at + r][c]);
#pragma unroll
            for (int x = 0; x < kTK; ++x)
              s[x][r] = fmaf(qv.x, kv[x].x,
                             fmaf(qv.y, kv[x].y, fmaf(qv.z, kv[x].z, fmaf(qv.w, kv[x].w, s[x][r]))));
          }
        }
        const unsigned there = __ballot_sync(0xffffffffu, cell >= 0);
#pragma unroll
        for (int x = 0; x < kTK; ++x) {
          const int key = key_at + x * kKg;
#pragma unroll
          for (int r = 0; r < kTR; ++r)
            s[x][r] = (there >> key) & 1 ? max_nan(s[x][r] * p.scale_log2, kLowestScore) : -INFINITY;
          st_vec<kTR>(&sm.p[warp][key][row_at], s[x]);
        }
        slice_sync();
      }
      copy(kc, kw, D + 4, next);
      if (work) {
        // keys of this warp that row `mine` sees, one bit each
        uint32_t see = 0xffffffffu;
        if (kTree) {
          const int from = first - part.seq.base;
          uint32_t lo = 0, hi = 0;
          if (tree != nullptr && from > -kKeys) {
            lo = tree_word(tree, p.tree_words, from >> 5);
            hi = tree_word(tree, p.tree_words, (from >> 5) + 1);
          }
          see = tree_window(lo, hi, from);
        }
        // row `mine`, keys lane / RP, + kPer, ...
        float x[RP], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          const int j = i * kPer + lane / RP;
          x[i] = (kTree ? (see >> j) & 1u : first + j < lim) ? sm.p[warp][j][mine] : -INFINITY;
          top = fmaxf(top, x[i]);
        }
#pragma unroll
        for (int o = RP; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m, top), use = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2_approx(m - use);
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          const float pr = ex2_approx(x[i] - use);
          sum += pr;
          sm.p[warp][i * kPer + lane / RP][mine] = pr;
        }
        l = fmaf(l, alpha, sum);
        m = mn;
        if (lane < RP) sm.alpha[warp][lane] = alpha;
        cp_async_wait<1>();  // this tile's values
        slice_sync();
#pragma unroll
        for (int r = 0; r < kOR; ++r) {
          const float shrink = sm.alpha[warp][orow_at + r];
#pragma unroll
          for (int c = 0; c < kOC; ++c) acc[r][c] *= shrink;
        }
#pragma unroll 8
        for (int j = 0; j < kKeys; ++j) {
          float v[kOC], pr[kOR];
#pragma unroll
          for (int c = 0; c < kOC; c += kOV)
            ld_vec<kOV>(&sm.v[slice][j][c * kOg + col_at], v + c);
          ld_vec<kOR>(&sm.p[warp][j][orow_at], pr);
#pragma unroll
          for (int r = 0; r < kOR; ++r)
#pragma unroll
            for (int c = 0; c < kOC; ++c) acc[r][c] = fmaf(pr[r], v[c], acc[r][c]);
        }
        slice_sync();
      }
      copy(vc, vw, D, next);
      cell = next;
    }
    cp_async_wait<0>();
    // join the warps: each leaves its sums where its values were
    __syncwarp();
#pragma unroll
    for (int o = RP; o < 32; o *= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane < RP) {
      sm.m[warp][lane] = m;
      sm.l[warp][lane] = l;
    }
#pragma unroll
    for (int r = 0; r < kOR; ++r)
#pragma unroll
      for (int c = 0; c < kOC; c += kOV)
        st_vec<kOV>(vw + (set * RP + orow_at + r) * D + c * kOg + col_at, &acc[r][c]);
    __syncthreads();
    const bool split = paged_split(part);
    float *slot = split ? paged_slot_ptr(p, D, blockIdx.x, paged_slot(part)) : nullptr;
    if (threadIdx.x < kAll) {
      const int r = threadIdx.x, of = r / RP * kWarps, in = r % RP;  // the row's warps, its place there
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm.m[of + w][in]);
      const float use = mt == -INFINITY ? 0.f : mt;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(sm.m[of + w][in] - use);
        lt = fmaf(sm.l[of + w][in], f, lt);
        sm.f[of + w][in] = f;
      }
      sm.total[r] = mt == kLowestScore ? NAN : lt;
      if (split && sm.row[r] >= 0) {
        slot[p.rows * D + 2 * r] = mt;
        slot[p.rows * D + 2 * r + 1] = lt;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x * 4; e < kAll * D; e += kSets * kThreads * 4) {
      const int r = e / D;
      const long long row = sm.row[r];
      if (row < 0) continue;
      float o[4] = {0.f, 0.f, 0.f, 0.f}, v[4];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ld_cols(&sm.v[w][0][e], v);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = fmaf(v[c], sm.f[r / RP * kWarps + w][r % RP], o[c]);
      }
      if (split) {
        st_cols(slot + e, o);
      } else {
        const float lt = sm.total[r];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = lt == 0.f ? 0.f : o[c] / lt;
        st_cols(out + row + e % D, o);
      }
    }
    if (split) {
      if (part.t0 > 0) {
        flags |= kPartContinues | (part.t1 == part.nt ? kPartEnds : 0);
        mrow = part.seq.q0 + part.i0;
        mtokens = part.i1 - part.i0;
        mhead = part.h0;
        mheads = part.heads;
      } else {
        flags |= kPartBegins;
      }
    }
  }
  if (threadIdx.x == 0) {
    int32_t *meta = p.meta + static_cast<size_t>(blockIdx.x) * kPagedMeta;
    meta[kMetaFlags] = flags;
    meta[kMetaRow] = mrow;
    meta[kMetaTokens] = mtokens;
    meta[kMetaHead] = mhead;
    meta[kMetaHeads] = mheads;
  }
}

// A unit to join, as its second part's CTA c describes it.
struct Joined {
  int row0, tokens, h0, heads;
  int c, last;  // CTAs of its second part and of its last
  // false: CTA c holds no unit's second part.  (Whole warp; the words are loaded at
  // once, for the merge is a chain of loads.)
  __device__ __forceinline__ bool find(const PagedProblem &p, int c, int ctas, int lane) {
    const int32_t *meta = p.meta + static_cast<size_t>(c) * kPagedMeta;
    const int4 own = *reinterpret_cast<const int4 *>(meta);
    const int before = meta[kMetaFlags - kPagedMeta];
    int flags = p.meta[static_cast<size_t>(min(c + lane, ctas - 1)) * kPagedMeta + kMetaFlags];
    heads = meta[kMetaHeads];
    static_assert(kMetaFlags == 0 && kMetaRow == 1 && kMetaTokens == 2 && kMetaHead == 3, "int4");
    this->c = c;
    row0 = own.y;
    tokens = own.z;
    h0 = own.w;
    if (!(own.x & kPartContinues) || !(before & kPartBegins)) return false;
    last = c;
    for (int at = c;;) {
      const unsigned ends = __ballot_sync(0xffffffffu, (flags & kPartEnds) != 0);
      if (ends != 0) {
        last = min(at + __ffs(ends) - 1, ctas - 1);
        break;
      }
      if ((at += 32) >= ctas) break;
      flags = p.meta[static_cast<size_t>(min(at + lane, ctas - 1)) * kPagedMeta + kMetaFlags];
    }
    return true;
  }
};

// CTA (c, y): if CTA c + 1 of the attention kernel holds the second part of a unit,
// that unit's rows are joined from its parts (slot 1 of CTA c, slot 0 of those behind
// it), in the order of their keys.  The eight warps share a row, row y of the unit:
// each takes every eighth part, its lanes d / 32 columns each.  A unit may have as many
// parts as there are CTAs, and a warp that went through them alone would wait for
// memory over and over (13 of then 22 us of one token over 8192 keys, d 128; 16 now).
// With more than 8 rows kSide rows to a CTA: the CTAs, most of which have nothing to do, come in
// fewer turns (16 rows, 32 sequences of 500-2000, d 64: 37.9 -> 36.5 us; 8 rows: 24.6, 24.7; 4
// rows 15.0, 15.2).
constexpr int kMergeWarps = 8, kMergeThreads = kMergeWarps * 32;
template <typename T, int D, int kSide>
__global__ void __launch_bounds__(kMergeThreads)
    paged_merge_kernel(const PagedProblem p, int ctas) {
  constexpr int kC = D / 32;
  __shared__ float sums[kSide][kMergeWarps][D];
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Joined u;
  if (!u.find(p, c, ctas, lane)) return;
  float o[kSide][kC], m[kSide], l[kSide], use[kSide];
  int at[kSide];  // row in a slot
  T *to[kSide];   // nullptr: no row
#pragma unroll
  for (int s = 0; s < kSide; ++s) {
    const int r = blockIdx.y * kSide + s, h = r / p.tb, i = r - h * p.tb;
    const bool there = r < p.rows && h < u.heads && i < u.tokens;
    at[s] = there ? r : 0;
    to[s] = there ? static_cast<T *>(p.out) +
                        (static_cast<long long>(u.row0 + i) * p.H + u.h0 + h) * D + lane * kC
                  : nullptr;
    m[s] = -INFINITY;
    l[s] = 0.f;
#pragma unroll
    for (int e = 0; e < kC; ++e) o[s][e] = 0.f;
  }
  const size_t sums_at = static_cast<size_t>(p.rows) * D;  // (max, sum) of rows in a slot
  for (int k = c - 1 + lane; k <= u.last; k += 32) {
    const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0) + sums_at;
    float2 part[kSide];
#pragma unroll
    for (int s = 0; s < kSide; ++s) part[s] = *reinterpret_cast<const float2 *>(slot + 2 * at[s]);
#pragma unroll
    for (int s = 0; s < kSide; ++s) {
      const float mn = fmaxf(m[s], part[s].x), be = mn == -INFINITY ? 0.f : mn;
      l[s] = l[s] * ex2_approx(m[s] - be) + part[s].y * ex2_approx(part[s].x - be);
      m[s] = mn;
    }
  }
#pragma unroll
  for (int s = 0; s < kSide; ++s) {
    const float top = warp_max(m[s]);
    use[s] = top == -INFINITY ? 0.f : top;
    l[s] = warp_sum(l[s] * ex2_approx(m[s] - use[s]));
    if (top == kLowestScore) l[s] = NAN;
  }
#pragma unroll 2
  for (int k = c - 1 + warp; k <= u.last; k += kMergeWarps) {
    const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
    float part[kSide][kC], top[kSide];  // this lane's kC columns
#pragma unroll
    for (int s = 0; s < kSide; ++s) {
      top[s] = slot[sums_at + 2 * at[s]];
      ld_cols(slot + static_cast<size_t>(at[s]) * D + lane * kC, part[s]);
    }
#pragma unroll
    for (int s = 0; s < kSide; ++s) {
      const float f = ex2_approx(top[s] - use[s]);
#pragma unroll
      for (int e = 0; e < kC; ++e) o[s][e] = fmaf(part[s][e], f, o[s][e]);
    }
  }
#pragma unroll
  for (int s = 0; s < kSide; ++s) st_cols(&sums[s][warp][lane * kC], o[s]);
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kSide; ++s) {  // a warp to a row
    if (warp != s || to[s] == nullptr) continue;
    float x[kC];
#pragma unroll
    for (int e = 0; e < kC; ++e) x[e] = 0.f;
#pragma unroll
    for (int g = 0; g < kMergeWarps; ++g) {
      float part[kC];
      ld_cols(&sums[s][g][lane * kC], part);
#pragma unroll
      for (int e = 0; e < kC; ++e) x[e] += part[e];
    }
    const float inv = 1.f / l[s];
#pragma unroll
    for (int e = 0; e < kC; ++e) x[e] = l[s] == 0.f ? 0.f : x[e] * inv;
    st_cols(to[s], x);
  }
}

// All units to join of the many-query kernel, found by every CTA of the merge for itself, in
// blocks of 32 of their rows (the tokens and heads that there are, which lie apart in a slot),
// dealt out by warps.  (1208 CTAs, each for 32 rows of a slot that may hold a part, came in
// turns, most of them for nothing, with two parts in flight to a warp: one tree of 16 tokens
// over 8192 keys, 32 heads over 8, d 128: 32.7 us, 21.3 so; of 64 tokens 37.7, 26.0; 16 of 9-25
// over 1000-4096 50.0, 48.6.  The few-query kernel's units are more and smaller: 2 us slower so.)
// Where many units of all rows are cut it is a little slower than those CTAs were (8 chunks of up
// to 512 tokens, 1000-4096 keys: 75.4, 76.4); one CTA to an SM: 80.4, three 78.3, four 77.7.
constexpr int kMergeRowsCtas = 2;  // to an SM
struct JoinedList {
  static constexpr int kWords = kMergeWarps;  // CTAs, a bit each
  static constexpr int kBlocks = 256 / 32;    // 32 rows of a unit, at most
  Joined unit[kPagedManyMaxCtas];             // by the CTA of its second part
  uint16_t block[kPagedManyMaxCtas * kBlocks];  // kBlocks times the unit, and which of its blocks
  uint32_t begins[kWords], ends[kWords];
  int count[kWords];

  // How many blocks there are.
  __device__ __forceinline__ int find(const PagedProblem &p, int ctas) {
    static_assert(kPagedManyMaxCtas <= kMergeThreads, "a CTA to a thread");
    const int c = threadIdx.x, lane = c & 31, warp = c >> 5;
    int4 own = make_int4(0, 0, 0, 0);
    int heads = 0;
    if (c < ctas) {
      const int32_t *meta = p.meta + static_cast<size_t>(c) * kPagedMeta;
      own = *reinterpret_cast<const int4 *>(meta);
      heads = meta[kMetaHeads];
    }
    const unsigned b = __ballot_sync(0xffffffffu, (own.x & kPartBegins) != 0);
    const unsigned e = __ballot_sync(0xffffffffu, (own.x & kPartEnds) != 0);
    if (lane == 0) {
      begins[warp] = b;
      ends[warp] = e;
    }
    __syncthreads();
    const bool start = c > 0 && (own.x & kPartContinues) != 0 &&
                       ((begins[(c - 1) >> 5] >> ((c - 1) & 31)) & 1) != 0;
    const int blocks = start ? min((own.z * heads + 31) / 32, kBlocks) : 0;
    int at = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += x;
    }
    if (lane == 31) count[warp] = at;
    at -= blocks;
    if (start) {
      int word = warp;
      uint32_t left = ends[word] & (0xffffffffu << lane);
      while (left == 0 && ++word < kWords) left = ends[word];
      Joined &u = unit[c];
      u.row0 = own.y;
      u.tokens = own.z;
      u.h0 = own.w;
      u.heads = heads;
      u.c = c;
      u.last = left != 0 ? word * 32 + __ffs(left) - 1 : c;
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      total += count[w];
      if (w < warp) at += count[w];
    }
    for (int x = 0; x < blocks; ++x) block[at + x] = static_cast<uint16_t>(c * kBlocks + x);
    __syncthreads();
    return total;
  }
};

// The same for the slots of paged_many_tc_kernel, [d / 4][rows][4] of up to 256 rows: a warp
// takes 32 of a unit's rows, one to a lane, and kC4 fours of columns, so that it reads 512
// bytes in a stretch, kDeep parts at once.
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    paged_merge_rows_kernel(const PagedProblem p, int ctas) {
  constexpr int kC4 = 4, kPieces = D / 4 / kC4, kDeep = 4;
  __shared__ JoinedList list;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tasks = list.find(p, ctas) * kPieces;
  // (neighbours in different CTAs)
  for (int task = warp * gridDim.x + blockIdx.x; task < tasks; task += kMergeWarps * gridDim.x) {
    const int block = list.block[task / kPieces], piece = task % kPieces;
    const Joined &u = list.unit[block / JoinedList::kBlocks];
    const int row = block % JoinedList::kBlocks * 32 + lane, h = row / u.tokens, i = row - h * u.tokens;
    if (h >= u.heads) continue;
    const int c = u.c, last = u.last, r = h * p.tb + i;  // row in a slot
    float o[kC4][4], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < kC4; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[e][x] = 0.f;
    for (int k0 = c - 1; k0 <= last; k0 += kDeep) {
      float part[kDeep][kC4][4];
      float2 ml[kDeep];
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        const int k = k0 + j;
        if (k > last) break;
        const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
        ml[j] = *reinterpret_cast<const float2 *>(slot + static_cast<size_t>(p.rows) * D + 2 * r);
#pragma unroll
        for (int e = 0; e < kC4; ++e)
          ld_cols(slot + (static_cast<size_t>(piece * kC4 + e) * p.rows + r) * 4, part[j][e]);
      }
#pragma unroll
      for (int j = 0; j < kDeep; ++j) {
        if (k0 + j > last) break;
        const float mn = fmaxf(m, ml[j].x), use = mn == -INFINITY ? 0.f : mn;
        const float older = ex2_approx(m - use), f = ex2_approx(ml[j].x - use);
        m = mn;
        l = fmaf(l, older, ml[j].y * f);
#pragma unroll
        for (int e = 0; e < kC4; ++e)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[e][x] = fmaf(o[e][x], older, part[j][e][x] * f);
      }
    }
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.out) +
                        (static_cast<long long>(u.row0 + i) * p.H + u.h0 + h) * D + piece * kC4 * 4;
    if (m == kLowestScore) l = NAN;
    const float inv = 1.f / l;
#pragma unroll
    for (int e = 0; e < kC4; e += 2) {
      uint32_t v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float a = o[e + x / 2][2 * (x % 2)], b = o[e + x / 2][2 * (x % 2) + 1];
        v[x] = l == 0.f ? 0u : pack_bf16x2(a * inv, b * inv);
      }
      st_global_v4(to + e * 4, make_uint4(v[0], v[1], v[2], v[3]));
    }
  }
}

template <typename... Args, typename... Given>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream,
                   Given... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int RP, bool kTree, int kSets = 1>
cudaError_t simt_as(const PagedProblem &p, int grid, cudaStream_t stream) {
  constexpr int kSmem = sizeof(Smem<D, kSets>);
  static_assert(kSmem <= 232448, "shared memory budget");
  const auto kernel = paged_simt_kernel<D, RP, kTree, kSets>;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(kernel), kSmem);
  if (e != cudaSuccess) return e;
  return launch(kernel, dim3(grid), kSets * kThreads, kSmem, stream, p);
}

template <int D, int RP>
cudaError_t simt(const PagedProblem &p, int grid, cudaStream_t stream) {
  return p.tree != nullptr ? simt_as<D, RP, true>(p, grid, stream)
                           : simt_as<D, RP, false>(p, grid, stream);
}

template <int D>
cudaError_t simt_rows(const PagedProblem &p, int grid, cudaStream_t stream) {
  const int R = p.hpu * p.tb;
  if (R <= 1) return simt<D, 1>(p, grid, stream);
  if (R <= 4) return simt<D, 4>(p, grid, stream);
  // (causal rows keep the order of their sums, which differs with the lanes to a row)
  if (R <= 8 && p.tree != nullptr) return simt_as<D, 8, true>(p, grid, stream);
  if (R <= kRows) return simt<D, 16>(p, grid, stream);
  if constexpr (D == 128) {
    if (R <= 2 * kRows && p.tree != nullptr) return simt_as<D, 16, true, 2>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_simt(const PagedProblem &p, int d, int grid, cudaStream_t stream) {
  return d == 64 ? simt_rows<64>(p, grid, stream) : simt_rows<128>(p, grid, stream);
}

namespace {

template <typename T, int D>
cudaError_t merge(const PagedProblem &p, int grid, cudaStream_t stream) {
  if (p.rows <= 8)
    return launch(paged_merge_kernel<T, D, 1>, dim3(grid - 1, p.rows), kMergeThreads, 0, stream, p,
                  grid);
  return launch(paged_merge_kernel<T, D, 2>, dim3(grid - 1, (p.rows + 1) / 2), kMergeThreads, 0, stream,
                p, grid);
}

template <int D>
cudaError_t merge_rows(const PagedProblem &p, int grid, int num_sms, cudaStream_t stream) {
  if (grid > kPagedManyMaxCtas) return cudaErrorInvalidValue;
  return launch(paged_merge_rows_kernel<D>, dim3(kMergeRowsCtas * num_sms), kMergeThreads, 0, stream,
                p, grid);
}

}  // namespace

cudaError_t launch_paged_merge(const PagedProblem &p, int d, int dtype, bool many, int grid,
                               int num_sms, cudaStream_t stream) {
  if (grid < 2) return cudaSuccess;
  if (many)
    return d == 64 ? merge_rows<64>(p, grid, num_sms, stream)
                   : merge_rows<128>(p, grid, num_sms, stream);
  if (dtype == 0)
    return d == 64 ? merge<float, 64>(p, grid, stream) : merge<float, 128>(p, grid, stream);
  return d == 64 ? merge<__nv_bfloat16, 64>(p, grid, stream)
                 : merge<__nv_bfloat16, 128>(p, grid, stream);
}

}  // namespace mha

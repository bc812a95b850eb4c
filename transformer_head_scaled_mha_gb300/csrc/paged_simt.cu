// Attention over a paged fp32 key/value cache on the CUDA cores (FFMA, no TF32), and
// the joining of split units that every paged attention kernel uses.
//
// A CTA of four warps walks its parts (paged.cuh): R <= 16 query rows of one
// key/value head against tiles of 128 keys.  Warp w takes keys 32 w .. 32 w + 31
// of each tile: scores with a key per lane (keys staged in shared memory, rows padded
// by 16 bytes so that lanes read without conflicts; queries broadcast), an online
// softmax with a row per lane, or 32 / R lanes to a row, through a small square of
// shared memory, then the value rows, each lane owning d / 32 output columns.  Keys and
// values are copied to shared memory without registers (cp.async): the next tile's keys
// while this one's softmax and values are worked on, its values while the next scores
// are, so a warp always has a tile in flight.  The warps' sums are joined once per part.
//
// Bound: few parts per CTA, so the time from launch to the first score and the code's
// own way into the instruction caches; hence one copy loop for both ends of a tile
// (the walk starts one tile early, with nothing to work on) and rows' places and
// limits in shared memory, found once.  Measured, with the merge: 8 sequences of 90-700
// keys, 5 tokens of 8 heads over 2, d 64: 17.5 us (44 with two tiles to a CTA and rows in
// registers); one token, 16 sequences of 1000-4000 keys, 32 heads over 8, d 128: 69 us,
// 4.8 TB/s; 4 tokens, 8 such sequences: 69 us, 2.4 TB/s.  Chunks and prompts take it as
// well, 16 rows at a time, each of which reads the keys again: 4 x 2048 tokens of 16 heads,
// d 64: 1391 us, 25 TFLOP/s; d 128: 3075 us, 22 TFLOP/s (0.3 of the CUDA cores' nominal
// 80), bound by the loads from shared memory (20 wavefronts to 64 FFMA in the score loop)
// and, at d 128, by one CTA of four warps to an SM.
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

template <int D>
struct Smem {
  float q[kRows][D];
  float k[kWarps][kKeys][D + 4];
  float v[kWarps][kKeys][D];          // at a part's end the warps' sums
  float p[kWarps][kKeys][kRows + 4];  // scores, then their powers
  float alpha[kWarps][kRows];         // what the older sums shrink to
  float m[kWarps][kRows], l[kWarps][kRows];
  float f[kWarps][kRows], total[kRows];  // the warps' weights when joined, and the sum
  long long row[kRows];                  // where a row's query and output begin (-1: no row)
  int lim[kRows];                        // keys below this are allowed
  long long scratch[40];
};

template <int D, int RP>
__global__ void __launch_bounds__(kThreads, 2) paged_simt_kernel(const __grid_constant__ PagedProblem p) {
  constexpr int kC = D / 32;  // output columns of a lane
  constexpr int kPer = 32 / RP;  // lanes to a row in the softmax
  static_assert(kRows <= kKeys, "a warp's sums fit where its values were");
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedSpan span = paged_span<kThreads>(p, blockIdx.x, gridDim.x, sm.scratch);
  PagedWalk walk;
  walk.begin(p, span);
  PagedPart part;
  int flags = 0, mrow = 0, mtokens = 0, mhead = 0, mheads = 0;
  const float *q = static_cast<const float *>(p.q);
  const float *kc = static_cast<const float *>(p.k), *vc = static_cast<const float *>(p.v);
  float *out = static_cast<float *>(p.out);
  float *kw = &sm.k[warp][0][0], *vw = &sm.v[warp][0][0];
  // copies a warp's 32 cache rows, one per lane's cell, zeros where there is none; 16
  // bytes per lane
  auto copy = [&](const float *cache, float *to, int stride, long long cell) {
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;  // lanes per row, rows at once
    const int c = (lane % kLanes) * 4;
#pragma unroll 4
    for (int j = 0; j < kKeys; j += kAtOnce) {
      const int row = j + lane / kLanes;
      const long long at = __shfl_sync(0xffffffffu, cell, row);
      cp_async16_or_zero(smem_addr(to + row * stride + c), cache + (at < 0 ? 0 : at) * D + c,
                         at >= 0);
    }
    cp_async_commit();
  };
  while (walk.next(p, part)) {
    __syncthreads();  // the part before has read q and the warps' sums
    if (threadIdx.x < RP) {
      const int r = threadIdx.x, h = r / p.tb, i = part.i0 + r - h * p.tb;
      sm.row[r] = h < part.heads && i < part.i1
                      ? (static_cast<long long>(part.seq.q0 + i) * p.H + part.h0 + h) * D
                      : -1;
      sm.lim[r] = paged_kv_end(part.seq, i + 1, p.causal);
    }
    __syncthreads();
    for (int e = threadIdx.x * 4; e < RP * D; e += kThreads * 4) {
      const long long row = sm.row[e / D];
      *reinterpret_cast<float4 *>(&sm.q[0][e]) =
          row >= 0 ? *reinterpret_cast<const float4 *>(q + row + e % D) : make_float4(0, 0, 0, 0);
    }
    const int mine = lane % RP, lim = sm.lim[mine];  // this lane's row in the softmax
    float m = -INFINITY, l = 0.f;                    // ... its maximum, and its share of the sum
    float acc[RP][kC];
#pragma unroll
    for (int r = 0; r < RP; ++r)
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[r][c] = 0.f;
    __syncthreads();
    long long cell = -1;
#pragma unroll 1
    for (int t = part.t0 - 1; t < part.t1; ++t) {
      const bool work = t >= part.t0;
      const int first = t * kPagedTile + warp * kKeys;  // this warp's keys
      // the next tile's cache row, one per lane (-1: none)
      const int ahead = first + kPagedTile + lane;
      const long long next = t + 1 < part.t1 && ahead < part.kv_end
                                 ? paged_cell(p.batch, part.b, ahead, part.kv, p.Hkv)
                                 : -1;
      if (work) {
        cp_async_wait<1>();  // this tile's keys (its values may be on their way)
        __syncwarp();
        float s[RP];
#pragma unroll
        for (int r = 0; r < RP; ++r) s[r] = 0.f;
#pragma unroll 2
        for (int c = 0; c < D; c += 4) {
          const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[warp][lane][c]);
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[r][c]);
            s[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[r]))));
          }
        }
#pragma unroll
        for (int r = 0; r < RP; ++r)
          sm.p[warp][lane][r] =
              cell >= 0 ? max_nan(s[r] * p.scale_log2, kLowestScore) : -INFINITY;
        __syncwarp();
      }
      copy(kc, kw, D + 4, next);
      if (work) {
        // row `mine`, keys lane / RP, + kPer, ...
        float x[RP], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int i = 0; i < RP; ++i) {
          const int j = i * kPer + lane / RP;
          x[i] = first + j < lim ? sm.p[warp][j][mine] : -INFINITY;
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
        __syncwarp();
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float shrink = sm.alpha[warp][r];
#pragma unroll
          for (int c = 0; c < kC; ++c) acc[r][c] *= shrink;
        }
#pragma unroll 4
        for (int j = 0; j < kKeys; ++j) {
          float v[kC];
#pragma unroll
          for (int c = 0; c < kC; ++c) v[c] = sm.v[warp][j][c * 32 + lane];
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            const float pr = sm.p[warp][j][r];
#pragma unroll
            for (int c = 0; c < kC; ++c) acc[r][c] = fmaf(pr, v[c], acc[r][c]);
          }
        }
        __syncwarp();
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
    for (int r = 0; r < RP; ++r)
#pragma unroll
      for (int c = 0; c < kC; ++c) vw[r * D + c * 32 + lane] = acc[r][c];
    __syncthreads();
    const bool split = paged_split(part);
    float *slot = split ? paged_slot_ptr(p, D, blockIdx.x, paged_slot(part)) : nullptr;
    if (threadIdx.x < RP) {
      const int r = threadIdx.x;
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm.m[w][r]);
      const float use = mt == -INFINITY ? 0.f : mt;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(sm.m[w][r] - use);
        lt = fmaf(sm.l[w][r], f, lt);
        sm.f[w][r] = f;
      }
      sm.total[r] = mt == kLowestScore ? NAN : lt;
      if (split && sm.row[r] >= 0) {
        slot[p.rows * D + 2 * r] = mt;
        slot[p.rows * D + 2 * r + 1] = lt;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x * 4; e < RP * D; e += kThreads * 4) {
      const int r = e / D;
      const long long row = sm.row[r];
      if (row < 0) continue;
      float o[4] = {0.f, 0.f, 0.f, 0.f}, v[4];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ld_cols(&sm.v[w][0][e], v);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = fmaf(v[c], sm.f[w][r], o[c]);
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
  int last;  // CTA of its last part
  // false: CTA c holds no unit's second part.  (Whole warp; the words are loaded at
  // once, for the merge is a chain of loads.)
  __device__ __forceinline__ bool find(const PagedProblem &p, int c, int ctas, int lane) {
    const int32_t *meta = p.meta + static_cast<size_t>(c) * kPagedMeta;
    const int4 own = *reinterpret_cast<const int4 *>(meta);
    const int before = meta[kMetaFlags - kPagedMeta];
    int flags = p.meta[static_cast<size_t>(min(c + lane, ctas - 1)) * kPagedMeta + kMetaFlags];
    heads = meta[kMetaHeads];
    static_assert(kMetaFlags == 0 && kMetaRow == 1 && kMetaTokens == 2 && kMetaHead == 3, "int4");
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
constexpr int kMergeWarps = 8;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    paged_merge_kernel(const PagedProblem p, int ctas) {
  constexpr int kC = D / 32;
  __shared__ float sums[kMergeWarps][D];
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Joined u;
  if (!u.find(p, c, ctas, lane)) return;
  const int r = blockIdx.y, h = r / p.tb, i = r - h * p.tb;
  if (h >= u.heads || i >= u.tokens) return;
  float o[kC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < kC; ++e) o[e] = 0.f;
  const size_t ml = static_cast<size_t>(p.rows) * D + 2 * r;  // (max, sum) in a slot
  for (int k = c - 1 + lane; k <= u.last; k += 32) {
    const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
    const float mk = slot[ml], lk = slot[ml + 1];
    const float mn = fmaxf(m, mk), to = mn == -INFINITY ? 0.f : mn;
    l = l * ex2_approx(m - to) + lk * ex2_approx(mk - to);
    m = mn;
  }
  const float top = warp_max(m), use = top == -INFINITY ? 0.f : top;
  l = warp_sum(l * ex2_approx(m - use));
  if (top == kLowestScore) l = NAN;
#pragma unroll 4
  for (int k = c - 1 + warp; k <= u.last; k += kMergeWarps) {
    const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
    const float f = ex2_approx(slot[ml] - use);
    float part[kC];  // this lane's kC columns
    ld_cols(slot + static_cast<size_t>(r) * D + lane * kC, part);
#pragma unroll
    for (int e = 0; e < kC; ++e) o[e] = fmaf(part[e], f, o[e]);
  }
  st_cols(&sums[warp][lane * kC], o);
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int e = 0; e < kC; ++e) o[e] = 0.f;
#pragma unroll
  for (int g = 0; g < kMergeWarps; ++g) {
    float part[kC];
    ld_cols(&sums[g][lane * kC], part);
#pragma unroll
    for (int e = 0; e < kC; ++e) o[e] += part[e];
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < kC; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
  st_cols(static_cast<T *>(p.out) + (static_cast<long long>(u.row0 + i) * p.H + u.h0 + h) * D +
              lane * kC,
          o);
}

// The same for the slots of paged_many_tc_kernel, [d / 4][rows][4] of up to 256 rows and
// few parts: CTA (c, y) takes rows 32 y + lane, warp w an eighth of the columns, so that
// a warp reads 512 bytes in a stretch.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
    paged_merge_rows_kernel(const PagedProblem p, int ctas) {
  constexpr int kC4 = D / 4 / kMergeWarps;  // fours of columns of a thread
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Joined u;
  if (!u.find(p, c, ctas, lane)) return;
  const int r = blockIdx.y * 32 + lane, h = r / p.tb, i = r - h * p.tb;
  if (r >= p.rows || h >= u.heads || i >= u.tokens) return;
  float o[kC4][4], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < kC4; ++e)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[e][x] = 0.f;
#pragma unroll 2
  for (int k = c - 1; k <= u.last; ++k) {
    const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
    float part[kC4][4];
#pragma unroll
    for (int e = 0; e < kC4; ++e)
      ld_cols(slot + (static_cast<size_t>(warp * kC4 + e) * p.rows + r) * 4, part[e]);
    const float2 ml = *reinterpret_cast<const float2 *>(slot + static_cast<size_t>(p.rows) * D + 2 * r);
    const float mn = fmaxf(m, ml.x), use = mn == -INFINITY ? 0.f : mn;
    const float older = ex2_approx(m - use), f = ex2_approx(ml.x - use);
    m = mn;
    l = fmaf(l, older, ml.y * f);
#pragma unroll
    for (int e = 0; e < kC4; ++e)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[e][x] = fmaf(o[e][x], older, part[e][x] * f);
  }
  __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.out) +
                      (static_cast<long long>(u.row0 + i) * p.H + u.h0 + h) * D + warp * kC4 * 4;
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

template <int D, int RP>
cudaError_t simt(const PagedProblem &p, int grid, cudaStream_t stream) {
  const cudaError_t e = set_smem_once(reinterpret_cast<const void *>(paged_simt_kernel<D, RP>),
                                      sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  return launch(paged_simt_kernel<D, RP>, dim3(grid), kThreads, sizeof(Smem<D>), stream, p);
}

template <int D>
cudaError_t simt_rows(const PagedProblem &p, int grid, cudaStream_t stream) {
  const int R = p.hpu * p.tb;
  if (R <= 1) return simt<D, 1>(p, grid, stream);
  if (R <= 4) return simt<D, 4>(p, grid, stream);
  return simt<D, 16>(p, grid, stream);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedProblem &p, int d, int grid, cudaStream_t stream) {
  if (p.hpu * p.tb > kRows) return cudaErrorInvalidValue;
  return d == 64 ? simt_rows<64>(p, grid, stream) : simt_rows<128>(p, grid, stream);
}

namespace {

template <typename T, int D>
cudaError_t merge(const PagedProblem &p, int grid, cudaStream_t stream) {
  return launch(paged_merge_kernel<T, D>, dim3(grid - 1, p.rows), kMergeWarps * 32, 0, stream, p,
                grid);
}

template <int D>
cudaError_t merge_rows(const PagedProblem &p, int grid, cudaStream_t stream) {
  return launch(paged_merge_rows_kernel<D>, dim3(grid - 1, (p.rows + 31) / 32), kMergeWarps * 32, 0,
                stream, p, grid);
}

}  // namespace

cudaError_t launch_paged_merge(const PagedProblem &p, int d, int dtype, bool many, int grid,
                               cudaStream_t stream) {
  if (grid < 2) return cudaSuccess;
  if (many) return d == 64 ? merge_rows<64>(p, grid, stream) : merge_rows<128>(p, grid, stream);
  if (dtype == 0)
    return d == 64 ? merge<float, 64>(p, grid, stream) : merge<float, 128>(p, grid, stream);
  return d == 64 ? merge<__nv_bfloat16, 64>(p, grid, stream)
                 : merge<__nv_bfloat16, 128>(p, grid, stream);
}

}  // namespace mha

// Attention over a paged key/value cache on the CUDA cores (FFMA, no TF32), and
// the joining of split units that every paged attention kernel uses.
//
// A CTA of four warps walks its parts (paged.cuh): R <= 16 query rows of one
// key/value head against tiles of 128 keys.  Warp w takes keys 32 w .. 32 w + 31
// of each tile, a key per lane: scores of all R rows against the lane's key
// (keys staged in shared memory, rows padded by 16 bytes so that lanes read
// without conflicts; queries broadcast), an online softmax per warp, then the
// value rows, each lane owning d / 32 output columns.  The warps' sums are
// joined once per part.
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

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_as(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16 *p, float v) { *p = __float2bfloat16(v); }

template <int D>
struct Smem {
  float q[kRows][D];
  float k[kWarps][kKeys][D + 4];  // later the warps' sums
  float p[kWarps][kKeys][kRows];
  float m[kWarps][kRows], l[kWarps][kRows];
  long long scratch[40];
};

template <typename T, int D, int RP>
__global__ void __launch_bounds__(kThreads) paged_simt_kernel(const PagedProblem p) {
  constexpr int kC = D / 32;  // output columns of a lane
  static_assert(sizeof(float) * kRows * D <= sizeof(float) * kKeys * (D + 4), "warp sums fit");
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const PagedSpan span = paged_span<kThreads>(p, blockIdx.x, gridDim.x, sm.scratch);
  PagedWalk walk;
  walk.begin(p, span);
  PagedPart part;
  int flags = 0, mseq = 0, mtok = 0, mhead = 0;
  const T *kc = static_cast<const T *>(p.k), *vc = static_cast<const T *>(p.v);
  T *out = static_cast<T *>(p.out);
  while (walk.next(p, part)) {
    __syncthreads();  // the part before has read q and the warps' sums
    for (int e = threadIdx.x; e < RP * D; e += kThreads) {
      const int r = e / D, c = e - r * D;
      const int h = r / p.tb, i = part.i0 + r % p.tb;
      float x = 0.f;
      if (h < part.heads && i < part.i1)
        x = to_f32(static_cast<const T *>(
            p.q)[(static_cast<long long>(part.seq.q0 + i) * p.H + part.h0 + h) * D + c]);
      sm.q[r][c] = x;
    }
    __syncthreads();
    float m[RP], l[RP], acc[RP][kC];
    int lim[RP];  // keys below this are allowed
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[r][c] = 0.f;
      const int i = part.i0 + r % p.tb;
      lim[r] = paged_kv_end(part.seq, i + 1, p.causal);
    }
    for (int t = part.t0; t < part.t1; ++t) {
      const int key0 = t * kPagedTile + warp * kKeys;
      if (key0 >= part.kv_end) break;
      const int key = key0 + lane;
      const long long cell =
          key < part.kv_end ? paged_cell(p.batch, part.b, key, part.kv, p.Hkv) : -1;
      __syncwarp();
      // the warp's key rows, zeros where there is none
#pragma unroll 8
      for (int j = 0; j < kKeys; ++j) {
        const long long at = __shfl_sync(0xffffffffu, cell, j);
#pragma unroll
        for (int c = 0; c < kC; ++c)
          sm.k[warp][j][c * 32 + lane] = at >= 0 ? to_f32(kc[at * D + c * 32 + lane]) : 0.f;
      }
      __syncwarp();
      float s[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) s[r] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        const float4 kv = *reinterpret_cast<const float4 *>(&sm.k[warp][lane][c]);
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[r][c]);
          s[r] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[r]))));
        }
      }
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float x = cell >= 0 && key < lim[r] ? s[r] * p.scale_log2 : -INFINITY;
        const float mn = fmaxf(m[r], warp_max(x));
        const float use = mn == -INFINITY ? 0.f : mn;
        const float pr = ex2_approx(x - use);
        const float alpha = ex2_approx(m[r] - use);
        l[r] = l[r] * alpha + pr;
        m[r] = mn;
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[r][c] *= alpha;
        sm.p[warp][lane][r] = pr;
      }
      __syncwarp();
#pragma unroll 4
      for (int j = 0; j < kKeys; ++j) {
        const long long at = __shfl_sync(0xffffffffu, cell, j);
        float v[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) v[c] = at >= 0 ? to_f32(vc[at * D + c * 32 + lane]) : 0.f;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float pr = sm.p[warp][j][r];
#pragma unroll
          for (int c = 0; c < kC; ++c) acc[r][c] = fmaf(pr, v[c], acc[r][c]);
        }
      }
    }
    // join the warps: each leaves its sums where its keys were
    __syncwarp();
    float *mine = &sm.k[warp][0][0];
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      const float lw = warp_sum(l[r]);
      if (lane == 0) {
        sm.m[warp][r] = m[r];
        sm.l[warp][r] = lw;
      }
#pragma unroll
      for (int c = 0; c < kC; ++c) mine[r * D + c * 32 + lane] = acc[r][c];
    }
    __syncthreads();
    const bool split = paged_split(part);
    float *slot = split ? paged_slot_ptr(p, D, blockIdx.x, paged_slot(part)) : nullptr;
    for (int e = threadIdx.x; e < RP * D; e += kThreads) {
      const int r = e / D, c = e - r * D;
      const int h = r / p.tb, i = part.i0 + r % p.tb;
      if (h >= part.heads || i >= part.i1) continue;
      float mt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, sm.m[w][r]);
      const float use = mt == -INFINITY ? 0.f : mt;
      float lt = 0.f, o = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_approx(sm.m[w][r] - use);
        lt = fmaf(sm.l[w][r], f, lt);
        o = fmaf(sm.k[w][0][r * D + c], f, o);
      }
      if (split) {
        slot[r * D + c] = o;
        if (c == 0) {
          slot[p.rows * D + 2 * r] = mt;
          slot[p.rows * D + 2 * r + 1] = lt;
        }
      } else {
        store_as(out + (static_cast<long long>(part.seq.q0 + i) * p.H + part.h0 + h) * D + c,
                 lt > 0.f ? o / lt : 0.f);
      }
    }
    if (split) {
      if (part.t0 > 0) {
        flags |= kPartContinues | (part.t1 == part.nt ? kPartEnds : 0);
        mseq = part.b;
        mtok = part.i0;
        mhead = part.h0;
      } else {
        flags |= kPartBegins;
      }
    }
  }
  if (threadIdx.x == 0) {
    int32_t *meta = p.meta + static_cast<size_t>(blockIdx.x) * kPagedMeta;
    meta[kMetaFlags] = flags;
    meta[kMetaSeq] = mseq;
    meta[kMetaTok] = mtok;
    meta[kMetaHead] = mhead;
  }
}

// CTA (c, y): if CTA c + 1 of the attention kernel holds the second part of a unit,
// rows y, y + gridDim.y, ... of that unit are joined from its parts, in the order
// of their keys.  A unit may have as many parts as there are CTAs, so lanes look at
// different parts for the last part, the maximum and the sum, and groups of D
// threads take every kGroups-th part of the output; a loop over the parts one
// after the other would wait for memory once per part (13 of the 22 us of one
// token over 8192 keys, d 128).
constexpr int kMergeThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedProblem p, int ctas) {
  constexpr int kGroups = kMergeThreads / D;
  __shared__ float sums[kGroups][D];
  griddep_launch_dependents();
  griddep_wait();
  const int c = blockIdx.x + 1;
  const int32_t *meta = p.meta + static_cast<size_t>(c) * kPagedMeta;
  if (!(meta[kMetaFlags] & kPartContinues) || !(meta[kMetaFlags - kPagedMeta] & kPartBegins)) return;
  const int lane = threadIdx.x & 31;
  const int col = threadIdx.x % D, group = threadIdx.x / D;
  int last = c;  // the parts are slot 1 of CTA c - 1 and slot 0 of CTAs c .. last
  for (int at = c; at < ctas; at += 32) {
    const int k = min(at + lane, ctas - 1);
    const unsigned ends = __ballot_sync(
        0xffffffffu, (p.meta[static_cast<size_t>(k) * kPagedMeta + kMetaFlags] & kPartEnds) != 0);
    if (ends != 0) {
      last = min(at + __ffs(ends) - 1, ctas - 1);
      break;
    }
  }
  const PagedSeq seq = paged_seq(p.batch, meta[kMetaSeq]);
  const int i0 = meta[kMetaTok], h0 = meta[kMetaHead];
  const int heads = min(p.hpu, p.group - h0 % p.group);
  for (int r = blockIdx.y; r < p.rows; r += gridDim.y) {
    const int h = r / p.tb, i = i0 + r % p.tb;
    if (h >= heads || i >= seq.n) continue;
    const size_t ml = static_cast<size_t>(p.rows) * D + 2 * r;  // (max, sum) of the row in a slot
    float m = -INFINITY, l = 0.f;
    for (int k = c - 1 + lane; k <= last; k += 32) {
      const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
      const float mk = slot[ml], lk = slot[ml + 1];
      const float mn = fmaxf(m, mk), use = mn == -INFINITY ? 0.f : mn;
      l = l * ex2_approx(m - use) + lk * ex2_approx(mk - use);
      m = mn;
    }
    const float top = warp_max(m), use = top == -INFINITY ? 0.f : top;
    l = warp_sum(l * ex2_approx(m - use));
    float o = 0.f;
#pragma unroll 4
    for (int k = c - 1 + group; k <= last; k += kGroups) {
      const float *slot = paged_slot_ptr(p, D, k, k < c ? 1 : 0);
      o = fmaf(slot[static_cast<size_t>(r) * D + col], ex2_approx(slot[ml] - use), o);
    }
    sums[group][col] = o;
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < kGroups; ++g) o += sums[g][col];
      store_as(static_cast<T *>(p.out) +
                   (static_cast<long long>(seq.q0 + i) * p.H + h0 + h) * D + col,
               l > 0.f ? o / l : 0.f);
    }
    __syncthreads();
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

template <typename T, int D, int RP>
cudaError_t simt(const PagedProblem &p, int grid, cudaStream_t stream) {
  const cudaError_t e = set_smem_once(
      reinterpret_cast<const void *>(paged_simt_kernel<T, D, RP>), sizeof(Smem<D>));
  if (e != cudaSuccess) return e;
  return launch(paged_simt_kernel<T, D, RP>, dim3(grid), kThreads, sizeof(Smem<D>), stream, p);
}

template <typename T, int D>
cudaError_t simt_rows(const PagedProblem &p, int grid, cudaStream_t stream) {
  const int R = p.hpu * p.tb;
  if (R <= 1) return simt<T, D, 1>(p, grid, stream);
  if (R <= 4) return simt<T, D, 4>(p, grid, stream);
  return simt<T, D, 16>(p, grid, stream);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedProblem &p, int d, int dtype, int grid,
                              cudaStream_t stream) {
  if (p.hpu * p.tb > kRows) return cudaErrorInvalidValue;
  if (dtype == 0)
    return d == 64 ? simt_rows<float, 64>(p, grid, stream) : simt_rows<float, 128>(p, grid, stream);
  return d == 64 ? simt_rows<__nv_bfloat16, 64>(p, grid, stream)
                 : simt_rows<__nv_bfloat16, 128>(p, grid, stream);
}

cudaError_t launch_paged_merge(const PagedProblem &p, int d, int dtype, int grid,
                               cudaStream_t stream) {
  if (grid < 2) return cudaSuccess;
  const dim3 g(grid - 1, p.rows < 16 ? p.rows : 16);
  if (dtype == 0)
    return d == 64 ? launch(paged_merge_kernel<float, 64>, g, kMergeThreads, 0, stream, p, grid)
                   : launch(paged_merge_kernel<float, 128>, g, kMergeThreads, 0, stream, p, grid);
  return d == 64 ? launch(paged_merge_kernel<__nv_bfloat16, 64>, g, kMergeThreads, 0, stream, p, grid)
                 : launch(paged_merge_kernel<__nv_bfloat16, 128>, g, kMergeThreads, 0, stream, p, grid);
}

}  // namespace mha

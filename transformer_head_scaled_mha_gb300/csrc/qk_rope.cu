// Per-head RMS norm and position rotation of query and key rows, their
// gradients, and the same on the way into a paged key/value cache.
//
// A row is one head of one token, d = 64 or 128 elements.  Per row
//
//   n = x w / sqrt(mean x^2 + eps)          (skipped without a weight)
//   (y_a, y_b) = (n_a c - n_b s, n_a s + n_b c),  c, s = cos, sin(p f_i)
//
// Bound: HBM (about 10 flop per element against 2 x 2 bytes).  d * sizeof(T) / 16
// lanes hold a row, 16 bytes each, so a row is read and written once with wide
// accesses and its sums are shuffles within those lanes.  A CTA takes `tb` tokens
// and walks their heads; the angles of a token are formed once, into shared
// memory, and serve all its heads.
//
// Angles: with the frequency in turns as a 64-bit binary fraction F =
// frac(f / 2 pi) 2^64, the position times F modulo 2^64 is the angle's fraction of
// a turn for any 32-bit position, because whole turns fall off the top; only the
// last step to fp32 rounds (to 2^-25 of a turn).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;  // tokens of a CTA at most

template <typename T>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(uint4 r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(uint4 r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};

// A plain 16-byte load that the compiler may not move to the read-only path: a
// row may be overwritten in place.
__device__ __forceinline__ uint4 ld16(const void *p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// frequency i as a 64-bit fraction of a turn per position
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  const double t = static_cast<double>(f) * 0.15915494309189533577;  // 1 / (2 pi)
  return static_cast<unsigned long long>((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ float2 angle_cos_sin(int pos, unsigned long long fraction) {
  const unsigned long long a = static_cast<unsigned long long>(static_cast<long long>(pos)) * fraction;
  const int top = static_cast<int>(static_cast<unsigned>(a >> 32));  // [-1/2, 1/2) turn
  float s, c;
  sincospif(static_cast<float>(top) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c, s);
}

// Where a tensor's rows of one token lie: element offset of head 0, step per head.
struct Rows {
  long long base, step;
};
__device__ __forceinline__ Rows rows_of(int layout, int t, int heads, int L, int d) {
  if (layout == kLayoutBSHD) return {static_cast<long long>(t) * heads * d, d};
  const int b = t / L, l = t - b * L;
  return {(static_cast<long long>(b) * heads * L + l) * d, static_cast<long long>(L) * d};
}

// What one thread holds of the rotation: its kN elements' factors.  out = x * c +
// partner * s, the sign of s included.
template <typename T, int D>
struct Lane {
  static constexpr int kN = Vec<T>::kN;
  float c[kN], s[kN];
  int partner;  // lane of the row's group that holds the other element of each pair
  bool on;      // its elements are rotated (rotary is a multiple of 16: all or none are)

  __device__ __forceinline__ void set(const float2 *cs, int col, int lane, int rotary, int style,
                                      bool back) {
    const int half = rotary >> 1;
    partner = lane;
    const int e0 = col * kN;
    on = e0 < rotary;
    if (style == kRopeHalves && on) partner = e0 < half ? lane + half / kN : lane - half / kN;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int e = e0 + i;
      c[i] = 1.f;
      s[i] = 0.f;
      if (on) {
        const bool first = style == kRopeHalves ? e < half : (e & 1) == 0;
        const float2 v = cs[style == kRopeHalves ? (e < half ? e : e - half) : e >> 1];
        c[i] = v.x;
        s[i] = first != back ? -v.y : v.y;
      }
    }
  }
  __device__ __forceinline__ void rotate(float (&x)[kN], int style) const {
    float o[kN];
    if (style == kRopeHalves) {
#pragma unroll
      for (int i = 0; i < kN; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], partner);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) o[i] = x[i ^ 1];
    }
    if (!on) return;
#pragma unroll
    for (int i = 0; i < kN; ++i) x[i] = fmaf(o[i], s[i], x[i] * c[i]);
  }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Norms and rotates `heads` rows of one token, every `hstep`-th from `h0`; all
// lanes of the warp call it (`live`: this lane's row group has a token).  kBatch
// rows are loaded before the first is stored.
template <typename T, int D, bool kCopy>
__device__ __forceinline__ void process_rows(const T *src, Rows in, T *dst, Rows to, int heads,
                                             int h0, int hstep, bool live, const T *weight,
                                             float eps, const Lane<T, D> &rot, int style,
                                             bool rotates, int col) {
  constexpr int kN = Vec<T>::kN, kLanes = D / kN, kBatch = 4;
  float w[kN];
  if (!kCopy && weight != nullptr) Vec<T>::unpack(ld16(weight + col * kN), w);
  const int rounds = (heads + hstep - 1) / hstep;  // the same for all lanes: shuffles inside
  for (int j = 0; j < rounds; j += kBatch) {
    uint4 raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + (j + i) * hstep;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (live && h < heads) raw[i] = ld16(src + in.base + h * in.step + col * kN);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + (j + i) * hstep;
      if (!kCopy) {
        if (j + i >= rounds) break;
        float x[kN];
        Vec<T>::unpack(raw[i], x);
        if (weight != nullptr) {
          float sq = 0.f;
#pragma unroll
          for (int e = 0; e < kN; ++e) sq = fmaf(x[e], x[e], sq);
          const float r = rsqrtf(row_sum<kLanes>(sq) * (1.f / D) + eps);
#pragma unroll
          for (int e = 0; e < kN; ++e) x[e] = x[e] * r * w[e];
        }
        if (rotates) rot.rotate(x, style);
        raw[i] = Vec<T>::pack(x);
      }
      if (live && h < heads) st_global_v4(dst + to.base + h * to.step + col * kN, raw[i]);
    }
  }
}

struct TokenInfo {
  long long cell;  // appending: cache row of head 0, or -1
  int pos;
  int live;
};

template <typename T, int D, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs a, int tb) {
  constexpr int kN = Vec<T>::kN, kLanes = D / kN, kSlots = kThreads / kLanes;
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ unsigned long long turns[D / 2];
  __shared__ TokenInfo info[kMaxTokens];
  griddep_launch_dependents();
  griddep_wait();
  const int t0 = blockIdx.x * tb;
  const int half = a.rotary >> 1;
  if (threadIdx.x >= kThreads - half) {
    const int f = threadIdx.x - (kThreads - half);
    turns[f] = turn_fraction(a.inv_freq[f]);
  }
  if (threadIdx.x < tb) {
    const int t = t0 + threadIdx.x;
    TokenInfo ti{-1, 0, 0};
    if (t < a.tokens) {
      if (kAppend) {
        const int b = paged_seq_of_row(a.batch, t);
        if (b >= 0) {
          // tokens up to the sequence's end count back from its length
          const int end = min(a.batch.q_starts[b + 1], a.tokens);
          ti.live = 1;
          ti.pos = max(a.batch.kv_lengths[b], 0) - (end - t);
          ti.cell = paged_cell(a.batch, b, ti.pos, 0, a.Hkv);
        }
      } else {
        ti.live = 1;
        ti.pos = a.positions != nullptr ? a.positions[t] : t % a.L;
      }
    }
    info[threadIdx.x] = ti;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tb * half; i += kThreads) {
    const int tok = i / half, f = i - tok * half;
    cs[tok][f] = angle_cos_sin(info[tok].pos, turns[f]);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int col = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int tok = slot % tb, h0 = slot / tb, hstep = kSlots / tb;
  const int t = t0 + tok;
  const bool live = info[tok].live != 0;
  Lane<T, D> rot;
  rot.set(cs[tok], col, lane, a.rotary, a.style, false);
  const int layout = kAppend ? kLayoutBSHD : a.layout;
  if (a.H > 0) {
    const Rows r = rows_of(layout, t, a.H, a.L, D);
    process_rows<T, D, false>(static_cast<const T *>(a.q), r, static_cast<T *>(a.q_out), r, a.H,
                              h0, hstep, live, static_cast<const T *>(a.q_weight), a.eps, rot,
                              a.style, half > 0, col);
  }
  if (a.Hkv > 0) {
    const Rows r = rows_of(layout, t, a.Hkv, a.L, D);
    Rows to = r;
    bool kept = live;
    if (kAppend) {
      kept = live && info[tok].cell >= 0;
      to.base = info[tok].cell * D;
      to.step = a.batch.layout == kLayoutBHSD ? static_cast<long long>(a.batch.page_size) * D : D;
    }
    process_rows<T, D, false>(static_cast<const T *>(a.k), r, static_cast<T *>(a.k_out), to, a.Hkv,
                              h0, hstep, kept, static_cast<const T *>(a.k_weight), a.eps, rot,
                              a.style, half > 0, col);
    if (kAppend)
      process_rows<T, D, true>(static_cast<const T *>(a.v), r, static_cast<T *>(a.v_out), to,
                               a.Hkv, h0, hstep, kept, nullptr, 0.f, rot, a.style, false, col);
  }
}

// Gradients of `heads` rows of one token; adds this lane's share of the weight's
// gradient to dw.
template <typename T, int D>
__device__ __forceinline__ void process_rows_bwd(const T *x_in, const T *dy, T *dx, Rows r,
                                                 int heads, int h0, int hstep, bool live,
                                                 const T *weight, float eps,
                                                 const Lane<T, D> &rot, int style, bool rotates,
                                                 int col, float (&dw)[Vec<T>::kN]) {
  constexpr int kN = Vec<T>::kN, kLanes = D / kN, kBatch = 2;
  float w[kN];
  const bool normed = weight != nullptr;
  if (normed) Vec<T>::unpack(ld16(weight + col * kN), w);
  const int rounds = (heads + hstep - 1) / hstep;
  for (int j = 0; j < rounds; j += kBatch) {
    uint4 rx[kBatch], rg[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + (j + i) * hstep;
      rx[i] = rg[i] = make_uint4(0, 0, 0, 0);
      if (live && h < heads) {
        const long long at = r.base + h * r.step + col * kN;
        rg[i] = ld16(dy + at);
        if (normed) rx[i] = ld16(x_in + at);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + (j + i) * hstep;
      if (j + i >= rounds) break;
      float g[kN];
      Vec<T>::unpack(rg[i], g);
      if (rotates) rot.rotate(g, style);
      if (normed) {
        float x[kN], sq = 0.f, dot = 0.f;
        Vec<T>::unpack(rx[i], x);
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          sq = fmaf(x[e], x[e], sq);
          dot = fmaf(g[e] * w[e], x[e], dot);
        }
        sq = row_sum<kLanes>(sq);
        dot = row_sum<kLanes>(dot);
        const float inv = rsqrtf(sq * (1.f / D) + eps);
        const float mean = dot * inv * (1.f / D);  // mean of (w g) (x inv)
        // an absent row adds nothing (its inv may be infinite)
        const float add = live && h < heads ? inv : 0.f;
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          dw[e] = fmaf(g[e], x[e] * add, dw[e]);
          g[e] = inv * (g[e] * w[e] - x[e] * inv * mean);
        }
      }
      if (live && h < heads) st_global_v4(dx + r.base + h * r.step + col * kN, Vec<T>::pack(g));
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const RopeArgs a, int tb) {
  constexpr int kN = Vec<T>::kN, kLanes = D / kN, kSlots = kThreads / kLanes;
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ unsigned long long turns[D / 2];
  __shared__ float sums[kSlots][D];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int col = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int tok = slot % tb, h0 = slot / tb, hstep = kSlots / tb;
  const int half = a.rotary >> 1;
  float dqw[kN], dkw[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) dqw[e] = dkw[e] = 0.f;
  if (threadIdx.x < half) turns[threadIdx.x] = turn_fraction(a.inv_freq[threadIdx.x]);
  __syncthreads();
  const int tiles = (a.tokens + tb - 1) / tb;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int t0 = tile * tb;
    for (int i = threadIdx.x; i < tb * half; i += kThreads) {
      const int k = i / half, f = i - k * half;
      const int t = min(t0 + k, a.tokens - 1);
      const int pos = a.positions != nullptr ? a.positions[t] : t % a.L;
      cs[k][f] = angle_cos_sin(pos, turns[f]);
    }
    __syncthreads();
    const int t = t0 + tok;
    const bool live = t < a.tokens;
    Lane<T, D> rot;
    rot.set(cs[tok], col, lane, a.rotary, a.style, true);
    if (a.H > 0)
      process_rows_bwd<T, D>(static_cast<const T *>(a.q), static_cast<const T *>(a.dq_out),
                             static_cast<T *>(a.q_out), rows_of(a.layout, t, a.H, a.L, D), a.H, h0,
                             hstep, live, static_cast<const T *>(a.q_weight), a.eps, rot, a.style,
                             half > 0, col, dqw);
    if (a.Hkv > 0)
      process_rows_bwd<T, D>(static_cast<const T *>(a.k), static_cast<const T *>(a.dk_out),
                             static_cast<T *>(a.k_out), rows_of(a.layout, t, a.Hkv, a.L, D), a.Hkv,
                             h0, hstep, live, static_cast<const T *>(a.k_weight), a.eps, rot,
                             a.style, half > 0, col, dkw);
    __syncthreads();  // cs is rewritten by the next tile
  }
  // this CTA's sums over its row slots, in a fixed order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.q_weight : a.k_weight) == nullptr) continue;
#pragma unroll
    for (int e = 0; e < kN; ++e) sums[slot][col * kN + e] = which == 0 ? dqw[e] : dkw[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
#pragma unroll
      for (int s = 0; s < kSlots; ++s) v += sums[s][threadIdx.x];
      a.partial[(static_cast<size_t>(blockIdx.x) * 2 + which) * D + threadIdx.x] = v;
    }
    __syncthreads();
  }
}

// dweight = sum of the CTAs' partial sums: CTA (x, y) takes columns 32 x .. + 31 of
// tensor y, warp w the rows w, w + 8, ...
__global__ void __launch_bounds__(256) rope_dweight_kernel(const float *partial, int rows, int d,
                                                           float *dq_weight, float *dk_weight) {
  __shared__ float sums[8][32];
  griddep_launch_dependents();
  griddep_wait();
  float *out = blockIdx.y == 0 ? dq_weight : dk_weight;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 4
  for (int r = warp; r < rows; r += 8) v += partial[(static_cast<size_t>(r) * 2 + blockIdx.y) * d + c];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][lane];
    out[c] = s;
  }
}

template <typename... Args, typename... Given>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t stream,
                   Given... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Tokens per CTA: four share a CTA when that still leaves every SM several CTAs.
int tokens_per_cta(int tokens, int num_sms) { return tokens >= 16 * num_sms ? kMaxTokens : 1; }

template <typename T, int D>
cudaError_t fwd(const RopeArgs &a, bool append, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_cta(a.tokens, num_sms);
  const dim3 grid((a.tokens + tb - 1) / tb);
  return append ? launch(rope_fwd_kernel<T, D, true>, grid, kThreads, stream, a, tb)
                : launch(rope_fwd_kernel<T, D, false>, grid, kThreads, stream, a, tb);
}

template <typename T, int D>
cudaError_t bwd(const RopeArgs &a, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_cta(a.tokens, num_sms);
  const int grid = std::min({(a.tokens + tb - 1) / tb, 4 * num_sms, kRopeBwdMaxCtas});
  cudaError_t e = cudaSuccess;
  if (grid > 0) e = launch(rope_bwd_kernel<T, D>, dim3(grid), kThreads, stream, a, tb);
  if (e == cudaSuccess && (a.dq_weight != nullptr || a.dk_weight != nullptr))
    e = launch(rope_dweight_kernel, dim3(D / 32, 2), 256, stream,
               static_cast<const float *>(a.partial), grid, D, a.dq_weight, a.dk_weight);
  return e;
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs &a, int d, int dtype, bool append, int num_sms,
                            cudaStream_t stream) {
  if (dtype == 0)
    return d == 64 ? fwd<float, 64>(a, append, num_sms, stream)
                   : fwd<float, 128>(a, append, num_sms, stream);
  return d == 64 ? fwd<__nv_bfloat16, 64>(a, append, num_sms, stream)
                 : fwd<__nv_bfloat16, 128>(a, append, num_sms, stream);
}

cudaError_t launch_rope_bwd(const RopeArgs &a, int d, int dtype, int num_sms, cudaStream_t stream) {
  if (dtype == 0)
    return d == 64 ? bwd<float, 64>(a, num_sms, stream) : bwd<float, 128>(a, num_sms, stream);
  return d == 64 ? bwd<__nv_bfloat16, 64>(a, num_sms, stream)
                 : bwd<__nv_bfloat16, 128>(a, num_sms, stream);
}

}  // namespace mha

// Per-head RMS norm and position rotation of query and key rows, their
// gradients, and the same on the way into a paged key/value cache.
//
// A row is one head of one token, d = 64 or 128 elements.  Per row
//
//   n = x w / sqrt(mean x^2 + eps)          (skipped without a weight)
//   (y_a, y_b) = (n_a c - n_b s, n_a s + n_b c),  c, s = cos, sin(p f_i)
//
// Bound: HBM (about 10 flop per element against 2 x 2 bytes).  d * sizeof(T) / 16
// lanes hold a row, 16 bytes each in two pieces, so a row is read and written once and its sums are shuffles within those lanes.  A CTA takes `tb` tokens
// and walks their heads, queries then keys (then values); the angles of a token are
// formed once, into shared memory, and serve all its heads.  The first rows are on
// their way before the angles are formed, and every row's load is issued kAhead
// rows before it is needed.
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
constexpr int kMaxTokens = 16;  // tokens of a CTA at most

// 16 bytes of a row, as a lane holds them: two pieces of 8 bytes.
template <typename T>
struct Vec;
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

// Plain loads that the compiler may not move to the read-only path: a row may be
// overwritten in place.
__device__ __forceinline__ uint4 ld8x2(const void *lo, const void *hi) {
  uint4 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(lo) : "memory");
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.z), "=r"(v.w) : "l"(hi) : "memory");
  return v;
}
__device__ __forceinline__ void st8x2(void *lo, void *hi, uint4 v) {
  asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(lo), "r"(v.x), "r"(v.y) : "memory");
  asm volatile("st.global.v2.b32 [%0], {%1, %2};" ::"l"(hi), "r"(v.z), "r"(v.w) : "memory");
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

// A lane's place in a row.  Both elements of a rotated pair belong to one lane:
// with MHA_ROPE_HALVES lane l of the rotated ones holds a piece of kN / 2 elements
// from each half, pair i being elements (i, i + kN / 2) of the lane's kN; otherwise
// the pieces lie side by side and pair i is (2 i, 2 i + 1).
template <typename T, int kStyle>
struct Place {
  static constexpr int kN = Vec<T>::kN, kPairs = kN / 2;
  int lo, hi;  // first elements of the two pieces
  int freq;    // first pair's frequency
  bool on;     // rotated (rotary is a multiple of 16: all of a lane's pairs are, or none)
  __device__ __forceinline__ Place(int col, int rotary) {
    on = col * kN < rotary;
    freq = col * kPairs;
    lo = kStyle == kRopeHalves && on ? col * kPairs : col * kN;
    hi = kStyle == kRopeHalves && on ? (rotary >> 1) + col * kPairs : col * kN + kPairs;
  }
  static __device__ __forceinline__ constexpr int a(int i) {
    return kStyle == kRopeHalves ? i : 2 * i;
  }
  static __device__ __forceinline__ constexpr int b(int i) {
    return kStyle == kRopeHalves ? i + kPairs : 2 * i + 1;
  }
  __device__ __forceinline__ uint4 load(const T *row) const { return ld8x2(row + lo, row + hi); }
  __device__ __forceinline__ void store(T *row, uint4 v) const { st8x2(row + lo, row + hi, v); }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct TokenInfo {
  long long cell;  // appending: cache row of head 0, or -1
  int pos;
  int live;
};

template <typename T, int D, int kStyle, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_fwd_kernel(const RopeArgs a, int tb) {
  using P = Place<T, kStyle>;
  constexpr int kN = Vec<T>::kN, kPairs = kN / 2, kLanes = D / kN, kSlots = kThreads / kLanes;
  constexpr int kAhead = 4;
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ unsigned long long turns[D / 2];
  __shared__ TokenInfo info[kMaxTokens];
  griddep_launch_dependents();
  const int col = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int tok = slot % tb, h0 = slot / tb, hstep = kSlots / tb;
  const int t0 = blockIdx.x * tb, t = t0 + tok;
  const P place(col, a.rotary);
  const int rounds_q = (a.H + hstep - 1) / hstep, rounds_k = (a.Hkv + hstep - 1) / hstep;
  const int rows = rounds_q + (kAppend ? 2 : 1) * rounds_k;
  const int layout = kAppend ? kLayoutBSHD : a.layout;
  const Rows rq = rows_of(layout, t, a.H, a.L, D), rk = rows_of(layout, t, a.Hkv, a.L, D);
  // element offsets of a slot's first row and between its rows
  const long long q0 = rq.base + h0 * rq.step, dq = hstep * rq.step;
  const long long k0 = rk.base + h0 * rk.step, dk = hstep * rk.step;
  // where the next row to load lies
  const T *src = static_cast<const T *>(a.q) + q0;
  int lj = 0, lh = h0;
  auto load = [&]() {
    if (lj == rounds_q || (kAppend && lj == rounds_q + rounds_k)) {
      src = static_cast<const T *>(lj == rounds_q ? a.k : a.v) + k0;
      lh = h0;
    }
    const bool q = lj < rounds_q;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (lj < rows && t < a.tokens && lh < (q ? a.H : a.Hkv)) v = place.load(src);
    src += q ? dq : dk;
    lh += hstep;
    ++lj;
    return v;
  };
  griddep_wait();
  uint4 raw[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) raw[i] = load();
  const int half = a.rotary >> 1;
  if (threadIdx.x >= kThreads - half) {
    const int f = threadIdx.x - (kThreads - half);
    turns[f] = turn_fraction(a.inv_freq[f]);
  }
  if (threadIdx.x < tb) {
    const int u = t0 + threadIdx.x;
    TokenInfo ti{-1, 0, 0};
    if (u < a.tokens) {
      if (kAppend) {
        const int b = paged_seq_of_row(a.batch, u);
        if (b >= 0) {
          // tokens up to the sequence's end count back from its length
          const int end = min(a.batch.q_starts[b + 1], a.tokens);
          ti.live = 1;
          ti.pos = max(a.batch.kv_lengths[b], 0) - (end - u);
          ti.cell = paged_cell(a.batch, b, ti.pos, 0, a.Hkv);
        }
      } else {
        ti.live = 1;
        ti.pos = a.positions != nullptr ? a.positions[u] : u % a.L;
      }
    }
    info[threadIdx.x] = ti;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tb * half; i += kThreads) {
    const int k = i / half, f = i - k * half;
    cs[k][f] = angle_cos_sin(info[k].pos, turns[f]);
  }
  __syncthreads();
  const bool live = info[tok].live != 0;
  const long long cell = info[tok].cell;
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const float2 v = place.on ? cs[tok][place.freq + i] : make_float2(1.f, 0.f);
    c[i] = v.x;
    s[i] = v.y;
  }
  // where the row goes, and this tensor's factors: y_a = r (a ca - b sb),
  // y_b = r (a sa + b cb), with the weight in them
  T *dst = static_cast<T *>(a.q_out) + q0;
  long long step = dq;
  int h = h0, heads = a.H;
  bool writes = live, normed = false, copies = false;
  float ca[kPairs], sb[kPairs], sa[kPairs], cb[kPairs];
  for (int j0 = 0; j0 < rows; j0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = j0 + i;
      if (j >= rows) break;
      uint4 v = raw[i];
      raw[i] = load();
      if (j == 0 || j == rounds_q || (kAppend && j == rounds_q + rounds_k)) {
        const bool q = j < rounds_q;
        copies = kAppend && j == rounds_q + rounds_k;
        if (!q) {
          h = h0;
          heads = a.Hkv;
          dst = static_cast<T *>(copies ? a.v_out : a.k_out);
          if (kAppend) {
            const long long per = a.batch.layout == kLayoutBHSD
                                      ? static_cast<long long>(a.batch.page_size) * D
                                      : D;
            writes = live && cell >= 0;
            dst += cell * D + h0 * per;
            step = hstep * per;
          } else {
            dst += k0;
            step = dk;
          }
        }
        const T *weight = static_cast<const T *>(q ? a.q_weight : a.k_weight);
        normed = weight != nullptr && !copies;
        float w[kN];
        if (normed) Vec<T>::unpack(place.load(weight), w);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const float wa = normed ? w[P::a(e)] : 1.f, wb = normed ? w[P::b(e)] : 1.f;
          ca[e] = c[e] * wa;
          sb[e] = s[e] * wb;
          sa[e] = s[e] * wa;
          cb[e] = c[e] * wb;
        }
      }
      if (!kAppend || !copies) {
        float y[kN];
        Vec<T>::unpack(v, y);
        float r = 1.f;
        if (normed) {
          float sq = 0.f;
#pragma unroll
          for (int e = 0; e < kN; ++e) sq = fmaf(y[e], y[e], sq);
          r = rsqrtf(row_sum<kLanes>(sq) * (1.f / D) + a.eps);
        }
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          const float ya = y[P::a(e)], yb = y[P::b(e)];
          float oa = ya * ca[e], ob = yb * cb[e];
          if (place.on) {  // outside the rotation an infinity must not meet a factor of 0
            oa = fmaf(-yb, sb[e], oa);
            ob = fmaf(ya, sa[e], ob);
          }
          y[P::a(e)] = oa * r;
          y[P::b(e)] = ob * r;
        }
        v = Vec<T>::pack(y);
      }
      if (writes && h < heads) place.store(dst, v);
      dst += step;
      h += hstep;
    }
  }
}

template <typename T, int D, int kStyle>
__global__ void __launch_bounds__(kThreads) rope_bwd_kernel(const RopeArgs a, int tb) {
  using P = Place<T, kStyle>;
  constexpr int kN = Vec<T>::kN, kPairs = kN / 2, kLanes = D / kN, kSlots = kThreads / kLanes;
  constexpr int kAhead = 2;
  __shared__ float2 cs[kMaxTokens][D / 2];
  __shared__ unsigned long long turns[D / 2];
  __shared__ float sums[kSlots][D];
  griddep_launch_dependents();
  griddep_wait();
  const int col = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const int tok = slot % tb, h0 = slot / tb, hstep = kSlots / tb;
  const int half = a.rotary >> 1;
  const P place(col, a.rotary);
  const int rounds_q = (a.H + hstep - 1) / hstep;
  const int rows = rounds_q + (a.Hkv + hstep - 1) / hstep;
  // this lane's share of the weights' gradients: of the tensor at hand, and of the other
  float dw[kN], other[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) dw[e] = other[e] = 0.f;
  if (threadIdx.x < half) turns[threadIdx.x] = turn_fraction(a.inv_freq[threadIdx.x]);
  const int tiles = (a.tokens + tb - 1) / tb;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int t0 = tile * tb, t = t0 + tok;
    const Rows rq = rows_of(a.layout, t, a.H, a.L, D), rk = rows_of(a.layout, t, a.Hkv, a.L, D);
    long long from = rq.base + h0 * rq.step, to = from;  // next row to load, to store
    int lj = 0, lh = h0, h = h0;
    uint4 raw_x[kAhead], raw_g[kAhead];
    auto load = [&](int i) {
      if (lj == rounds_q) {
        from = rk.base + h0 * rk.step;
        lh = h0;
      }
      const bool q = lj < rounds_q;
      raw_x[i] = raw_g[i] = make_uint4(0, 0, 0, 0);
      if (lj < rows && t < a.tokens && lh < (q ? a.H : a.Hkv)) {
        raw_g[i] = place.load(static_cast<const T *>(q ? a.dq_out : a.dk_out) + from);
        if ((q ? a.q_weight : a.k_weight) != nullptr)
          raw_x[i] = place.load(static_cast<const T *>(q ? a.q : a.k) + from);
      }
      from += hstep * (q ? rq.step : rk.step);
      lh += hstep;
      ++lj;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    __syncthreads();  // the tile before has read cs; turns are written
    for (int i = threadIdx.x; i < tb * half; i += kThreads) {
      const int k = i / half, f = i - k * half;
      const int u = min(t0 + k, a.tokens - 1);
      const int pos = a.positions != nullptr ? a.positions[u] : u % a.L;
      cs[k][f] = angle_cos_sin(pos, turns[f]);
    }
    __syncthreads();
    float c[kPairs], s[kPairs], w[kN];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 v = place.on ? cs[tok][place.freq + i] : make_float2(1.f, 0.f);
      c[i] = v.x;
      s[i] = v.y;
    }
    bool normed = false;
    auto turn = [&]() {
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float v = dw[e];
        dw[e] = other[e];
        other[e] = v;
      }
    };
    for (int j0 = 0; j0 < rows; j0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i;
        if (j >= rows) break;
        const bool q = j < rounds_q;
        if (j == rounds_q) {
          to = rk.base + h0 * rk.step;
          h = h0;
          turn();
        }
        if (j == 0 || j == rounds_q) {
          const T *weight = static_cast<const T *>(q ? a.q_weight : a.k_weight);
          normed = weight != nullptr;
          if (normed) Vec<T>::unpack(place.load(weight), w);
        }
        float g[kN], x[kN];
        Vec<T>::unpack(raw_g[i], g);
        Vec<T>::unpack(raw_x[i], x);
        load(i);
        const bool is = t < a.tokens && h < (q ? a.H : a.Hkv);
        if (place.on) {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const float ga = g[P::a(e)], gb = g[P::b(e)];
            g[P::a(e)] = fmaf(gb, s[e], ga * c[e]);
            g[P::b(e)] = fmaf(-ga, s[e], gb * c[e]);
          }
        }
        if (normed) {
          float sq = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            sq = fmaf(x[e], x[e], sq);
            dot = fmaf(g[e] * w[e], x[e], dot);
          }
          sq = row_sum<kLanes>(sq);
          dot = row_sum<kLanes>(dot);
          const float inv = rsqrtf(sq * (1.f / D) + a.eps);
          const float mean = dot * inv * (1.f / D);  // mean of (w g) (x inv)
          const float add = is ? inv : 0.f;  // an absent row adds nothing (its inv may be infinite)
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            dw[e] = fmaf(g[e], x[e] * add, dw[e]);
            g[e] = inv * (g[e] * w[e] - x[e] * inv * mean);
          }
        }
        if (is) place.store(static_cast<T *>(q ? a.q_out : a.k_out) + to, Vec<T>::pack(g));
        to += hstep * (q ? rq.step : rk.step);
        h += hstep;
      }
    }
    if (rounds_q < rows) turn();  // q's again
  }
  // this CTA's sums over its row slots, in a fixed order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.q_weight : a.k_weight) == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kN; ++e)
      sums[slot][(e < kPairs ? place.lo : place.hi) + e % kPairs] = which == 0 ? dw[e] : other[e];
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kSlots; ++k) v += sums[k][threadIdx.x];
      a.partial[(static_cast<size_t>(blockIdx.x) * 2 + which) * D + threadIdx.x] = v;
    }
  }
}

// dweight = sum of the CTAs' partial sums: CTA (x, y) takes columns 32 x .. + 31 of
// tensor y, warp w the rows w, w + 32, ...
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32)
    rope_dweight_kernel(const float *partial, int rows, int d, float *dq_weight, float *dk_weight) {
  __shared__ float sums[kSumWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  float *out = blockIdx.y == 0 ? dq_weight : dk_weight;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 8
  for (int r = warp; r < rows; r += kSumWarps)
    v += partial[(static_cast<size_t>(r) * 2 + blockIdx.y) * d + c];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) s += sums[w][lane];
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

// Tokens per CTA: more share a CTA, and its angles' latency, while a row slot has
// fewer than 8 rows and the SMs keep several CTAs each.
int tokens_per_cta(int tokens, int heads, int slots, int num_sms) {
  int tb = 1;
  while (tb < std::min(kMaxTokens, slots) && tb * heads < 8 * slots &&
         tokens / (2 * tb) >= 4 * num_sms)
    tb *= 2;
  return tb;
}

template <typename T, int D>
constexpr int slots() {
  return kThreads / (D / Vec<T>::kN);
}

template <typename T, int D, int kStyle>
cudaError_t fwd(const RopeArgs &a, bool append, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_cta(a.tokens, a.H + (append ? 2 : 1) * a.Hkv, slots<T, D>(), num_sms);
  const dim3 grid((a.tokens + tb - 1) / tb);
  return append ? launch(rope_fwd_kernel<T, D, kStyle, true>, grid, kThreads, stream, a, tb)
                : launch(rope_fwd_kernel<T, D, kStyle, false>, grid, kThreads, stream, a, tb);
}

template <typename T, int D, int kStyle>
cudaError_t bwd(const RopeArgs &a, int num_sms, cudaStream_t stream) {
  const int tb = tokens_per_cta(a.tokens, a.H + a.Hkv, slots<T, D>(), num_sms);
  const int grid = std::min({(a.tokens + tb - 1) / tb, 4 * num_sms, kRopeBwdMaxCtas});
  cudaError_t e = cudaSuccess;
  if (grid > 0) e = launch(rope_bwd_kernel<T, D, kStyle>, dim3(grid), kThreads, stream, a, tb);
  if (e == cudaSuccess && (a.dq_weight != nullptr || a.dk_weight != nullptr))
    e = launch(rope_dweight_kernel, dim3(D / 32, 2), kSumWarps * 32, stream,
               static_cast<const float *>(a.partial), grid, D, a.dq_weight, a.dk_weight);
  return e;
}

template <typename T, int D>
cudaError_t rope(const RopeArgs &a, int mode, int num_sms, cudaStream_t stream) {
  if (a.style == kRopeHalves)
    return mode < 2 ? fwd<T, D, kRopeHalves>(a, mode == 1, num_sms, stream)
                    : bwd<T, D, kRopeHalves>(a, num_sms, stream);
  return mode < 2 ? fwd<T, D, kRopeInterleaved>(a, mode == 1, num_sms, stream)
                  : bwd<T, D, kRopeInterleaved>(a, num_sms, stream);
}

// mode: 0 forward, 1 append, 2 backward
cudaError_t rope_of(const RopeArgs &a, int d, int dtype, int mode, int num_sms,
                    cudaStream_t stream) {
  if (dtype == 0)
    return d == 64 ? rope<float, 64>(a, mode, num_sms, stream)
                   : rope<float, 128>(a, mode, num_sms, stream);
  return d == 64 ? rope<__nv_bfloat16, 64>(a, mode, num_sms, stream)
                 : rope<__nv_bfloat16, 128>(a, mode, num_sms, stream);
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs &a, int d, int dtype, bool append, int num_sms,
                            cudaStream_t stream) {
  return rope_of(a, d, dtype, append ? 1 : 0, num_sms, stream);
}

cudaError_t launch_rope_bwd(const RopeArgs &a, int d, int dtype, int num_sms, cudaStream_t stream) {
  return rope_of(a, d, dtype, 2, num_sms, stream);
}

}  // namespace mha

// Per-head RMS norm and position rotation of query and key rows, their
// gradients, and the same on the way into a paged key/value cache.
//
// A row is one head of one token, d = 64 or 128 elements.  Per row
//
//   n = x w / sqrt(mean x^2 + eps)          (skipped without a weight)
//   (y_a, y_b) = (n_a c - n_b s, n_a s + n_b c),  c, s = cos, sin(p f_i)
//
// Bound: HBM (about 10 flop per element against 2 x 2 bytes), then the instructions
// issued per row.  d * sizeof(T) / 16 lanes hold a row, 16 bytes each in two pieces,
// so a row is read and written once and its sums are shuffles within those lanes;
// a warp holds 1, 2 or 4 rows at a time.  A warp takes one token, or a share of its
// rows, forms the token's angles once, in registers, and walks the token's heads,
// queries then keys (then values), four warp-rows in flight.  No shared memory and
// no barrier: what a CTA-wide table of angles costs in waiting and bookkeeping is
// more than computing an angle per lane and token.
//
// The backward reads two rows for each it writes and sums for the weights between
// them: its rows are copied ahead into shared memory (Ahead).
//
// Measured: forward, 4 x 8192 tokens of 16 + 16 heads, d 128: 90 us, 5.96 TB/s (0.88 of a
// copy's rate); appended prompts of 32 + 8 + 8 heads, d 128: 40.4 us (0.79); backward, 2 x
// 4096 tokens of 32 + 8 heads, d 128: 47 us (0.79).  fp32: forward, 2 x 8192 tokens of 16 +
// 16, d 128: 87 us (0.91); those prompts 73 us (0.88); that backward 82 us (0.90).  Few short
// rows to a token are bound by latency, with neither the issue slots (54%) nor DRAM (31%)
// full: 128 x 127 tokens of 8 + 8 heads, d 64, backward 28 us (0.53: a round at a time, its
// sums six shuffles behind one another, and 5 us before the first row and for the weights'
// last sums), forward 26 (0.38: two rounds of loads to a token's tensor).  256 trees of 64
// tokens of 8 + 8 + 8 heads appended: 22.7 us (0.66; 26.7 with a tensor's rows loaded after
// the one before was done), latency as well: a token's loads, lookups and stores follow one
// another, 20 warps to an SM, with DRAM 33% busy, the issue slots 57% while an SM works and 43%
// of the whole launch.  One loop over all tensors' rounds, six loads ahead, for any number of
// heads: 28.5, and prompts 53.
//
// Angles: with the frequency in turns as a 64-bit binary fraction F =
// frac(f / 2 pi) 2^64, the position times F modulo 2^64 is the angle's fraction of
// a turn for any 32-bit position, because whole turns fall off the top.  F is short of
// the fraction by less than 2^-64, the angle of the farthest position by 2^-33 of a turn;
// the step to fp32 drops less than 2^-32 and rounds to 2^-26 of a turn.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kFwdCtas = 3, kBwdCtas = 2;  // per SM
constexpr int kSlots = 4;                  // rounds of the backward in shared memory, per warp
constexpr int kSlotBytes = 1024;           // of a round: 16 of dy and 16 of x per lane

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

// Two fp32 in one 64-bit register, multiplied and added by one instruction: the
// backward's rows are bound by instructions issued (65 -> 59 us on 8192 tokens of
// 32 + 8 heads, d 128; the forward gains nothing and spills).  Subnormal values are
// kept.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

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

// 8 bytes to shared memory, without waiting; zeros unless `is`
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool is) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(is ? 8 : 0)
               : "memory");
}
// a lane's two pieces of 8 bytes, 256 apart
__device__ __forceinline__ uint4 lds8x2(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.z), "=r"(v.w) : "r"(at + 256) : "memory");
  return v;
}

// frac(f / 2 pi) 2^64, the fraction rounded down, for f = m 2^e, |f| < 2^20: m times
// 2^130 / (2 pi) in two words, shifted.  The second word carries the fraction's last bits
// for f > 2^-4: without it a position of 2^31 at f = 2^20 is off by up to 2^-18 of a turn.
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  constexpr unsigned long long k0 = 11743562013128004905ull, k1 = 18169587780923219392ull;
  const uint32_t bits = __float_as_uint(f);
  const int exp = (bits >> 23) & 255;
  const unsigned long long m = (bits & 0x7fffffu) | (exp != 0 ? 0x800000u : 0u);
  const int right = 2 - ((exp != 0 ? exp : 1) - 150);  // bits to drop of the 88 above k1's
  const unsigned long long carry = __umul64hi(m, k1), lo = m * k0 + carry;
  const unsigned long long hi = __umul64hi(m, k0) + (lo < carry ? 1 : 0);
  unsigned long long v = 0;  // (|f| from 2^28 on, infinities and NaN: no rotation)
  if (right >= 64) v = right < 128 ? hi >> (right - 64) : 0;
  else if (right > 0) v = (hi << (64 - right)) | (lo >> right);
  return (bits >> 31) != 0 ? 0 - v : v;
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

// How the kernels see the rotation: the two styles for any rotary_dim, and halves
// over the whole head, where the pieces' distance is a constant.
enum Style { kHalves = 0, kInterleaved = 1, kWholeHalves = 2 };

// A lane's place in a row, and its elements as kTwos packed twos of first elements a
// and of second elements b of its pairs.  Both elements of a rotated pair belong to
// one lane: with halves lane l of the rotated ones holds a piece of kN / 2 elements
// from each half, pair i being elements (i, i + kN / 2) of the lane's kN; otherwise
// the pieces lie side by side and pair i is (2 i, 2 i + 1).
template <typename T, int D, int kStyle>
struct Place {
  static constexpr int kN = Vec<T>::kN, kPairs = kN / 2, kTwos = kPairs / 2;
  int lo;     // first element of the first piece
  int apart;  // from there to the second piece
  int freq;   // first pair's frequency
  bool on;    // rotated (rotary is a multiple of 16: all of a lane's pairs are, or none)
  __device__ __forceinline__ Place(int col, int rotary) {
    on = kStyle == kWholeHalves || col * kN < rotary;
    freq = col * kPairs;
    lo = kStyle != kInterleaved && on ? col * kPairs : col * kN;
    apart = kStyle == kWholeHalves ? D / 2
                                   : (kStyle == kHalves && on ? rotary >> 1 : kPairs);
    if (kStyle == kInterleaved) apart = kPairs;
  }
  __device__ __forceinline__ uint4 load(const T *row) const {
    return ld8x2(row + lo, row + lo + apart);
  }
  __device__ __forceinline__ void store(T *row, uint4 v) const {
    st8x2(row + lo, row + lo + apart, v);
  }
  // which of the lane's elements pair i's are
  static __device__ __forceinline__ constexpr int a(int i) {
    return kStyle == kInterleaved ? 2 * i : i;
  }
  static __device__ __forceinline__ constexpr int b(int i) {
    return kStyle == kInterleaved ? 2 * i + 1 : i + kPairs;
  }
  // element of the row that a[i] (second: b[i]) holds
  __device__ __forceinline__ int element(int i, bool second) const {
    return kStyle == kInterleaved ? lo + 2 * i + second : lo + i + (second ? apart : 0);
  }
  static __device__ __forceinline__ void unpack(uint4 v, uint64_t (&a)[kTwos],
                                                uint64_t (&b)[kTwos]) {
    float x[kN];
    Vec<T>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < kTwos; ++i) {
      constexpr bool kSide = kStyle == kInterleaved;
      a[i] = kSide ? f2_pack(x[4 * i], x[4 * i + 2]) : f2_pack(x[2 * i], x[2 * i + 1]);
      b[i] = kSide ? f2_pack(x[4 * i + 1], x[4 * i + 3])
                   : f2_pack(x[kPairs + 2 * i], x[kPairs + 2 * i + 1]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const uint64_t (&a)[kTwos],
                                               const uint64_t (&b)[kTwos]) {
    float x[kN];
#pragma unroll
    for (int i = 0; i < kTwos; ++i) {
      constexpr bool kSide = kStyle == kInterleaved;
      f2_unpack(a[i], x[kSide ? 4 * i : 2 * i], x[kSide ? 4 * i + 2 : 2 * i + 1]);
      f2_unpack(b[i], x[kSide ? 4 * i + 1 : kPairs + 2 * i],
                x[kSide ? 4 * i + 3 : kPairs + 2 * i + 1]);
    }
    return Vec<T>::pack(x);
  }
};

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of a lane's pairs.  A warp's kGroups row groups need the same angles:
// each forms its share, and they pass them around.
template <typename T, int D>
struct Angles {
  static constexpr int kN = Vec<T>::kN, kPairs = kN / 2, kLanes = D / kN, kGroups = 32 / kLanes;
  static constexpr int kOwn = kPairs / kGroups;
  static_assert(kOwn >= 1, "a lane forms at least one angle");
  unsigned long long turns[kOwn];
  uint64_t c[kPairs / 2], s[kPairs / 2];
  // lanes outside the rotation keep angle 0
  __device__ __forceinline__ void frequencies(const float *inv_freq, int first, bool on, int group) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      turns[i] = on ? turn_fraction(inv_freq[first + group * kOwn + i]) : 0ull;
  }
  __device__ __forceinline__ void at(int pos, int col) {
    float2 own[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own[i] = angle_cos_sin(pos, turns[i]);
    float x[kPairs], y[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      x[i] = __shfl_sync(0xffffffffu, own[i % kOwn].x, (i / kOwn) * kLanes + col);
      y[i] = __shfl_sync(0xffffffffu, own[i % kOwn].y, (i / kOwn) * kLanes + col);
    }
#pragma unroll
    for (int i = 0; i < kPairs / 2; ++i) {
      c[i] = f2_pack(x[2 * i], x[2 * i + 1]);
      s[i] = f2_pack(y[2 * i], y[2 * i + 1]);
    }
  }
};

// Sequence of row t (whole warp): the last one that starts at or before it, -1 when
// the row belongs to none.  32 offsets are looked at a time; q_starts[lo] <= t <
// q_starts[hi] holds throughout, whatever the numbers.
__device__ __forceinline__ int seq_of_row(const PagedBatch &p, int t, int lane) {
  int lo = 0, hi = p.B;
  if (t < p.q_starts[0] || t >= p.q_starts[p.B]) return -1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < hi && p.q_starts[min(at, hi)] <= t);
    const int last = 31 - __clz(below | 1u);
    lo += last * step;
    hi = min(lo + step, hi);
  }
  return lo;
}

// A warp's work.  A token's rows come in rounds of kGroups heads: q's rounds, then
// k's, then, when appending, v's.  The warps take equal stretches of all tokens'
// rounds, so that a token count that does not fill the last pass over the SMs costs
// nothing; a warp forms the angles of each token that its stretch touches.
struct Stretch {
  long long at, end;
  __device__ __forceinline__ Stretch(long long total, int warp, int warps) {
    const long long each = total / warps, over = total % warps;
    at = each * warp + over * warp / warps;
    end = each * (warp + 1) + over * (warp + 1) / warps;
  }
  // the next token and its rounds [lo, hi) of `rounds`; false at the end
  __device__ __forceinline__ bool next(int rounds, int &token, int &lo, int &hi) {
    if (at >= end) return false;
    const long long t = at <= 0x7fffffff ? static_cast<int>(at) / rounds : at / rounds;
    token = static_cast<int>(t);
    lo = static_cast<int>(at - t * rounds);
    hi = static_cast<int>(min(static_cast<long long>(rounds), lo + (end - at)));
    at += hi - lo;
    return true;
  }
};

// What a token's rows of one tensor are multiplied by: y_a = r (a ca - b sb), y_b = r (a sa
// + b cb), the weight in the factors.
template <typename T, int D, int kStyle>
struct Factors {
  using P = Place<T, D, kStyle>;
  static constexpr int kN = P::kN, kPairs = P::kPairs;
  float ca[kPairs], sb[kPairs], sa[kPairs], cb[kPairs];
  bool normed;
  __device__ __forceinline__ void set(const Angles<T, D> &ang, const P &place, const T *weight) {
    normed = weight != nullptr;
    float w[kN];
    if (normed) Vec<T>::unpack(place.load(weight), w);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      float c0, c1, s0, s1;
      f2_unpack(ang.c[e / 2], c0, c1);
      f2_unpack(ang.s[e / 2], s0, s1);
      const float c = e % 2 == 0 ? c0 : c1, s = e % 2 == 0 ? s0 : s1;
      const float wa = normed ? w[P::a(e)] : 1.f, wb = normed ? w[P::b(e)] : 1.f;
      ca[e] = c * wa;
      sb[e] = s * wb;
      sa[e] = s * wa;
      cb[e] = c * wb;
    }
  }
  __device__ __forceinline__ uint4 apply(uint4 raw, const P &place, float eps) const {
    float y[kN];
    Vec<T>::unpack(raw, y);
    float r = 1.f;
    if (normed) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < kN; ++e) sq = fmaf(y[e], y[e], sq);
      r = rsqrtf(row_sum<Angles<T, D>::kLanes>(sq) * (1.f / D) + eps);
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
    return Vec<T>::pack(y);
  }
};

// Norms and rotates (or, kCopy, copies) rounds [from, to) of one tensor.  Row h lies
// at src + h * in and goes to dst + h * out.
template <typename T, int D, int kStyle, bool kCopy>
__device__ __forceinline__ void fwd_rows(const T *src, long long in, T *dst, long long out,
                                         int heads, int from, int to, int group, bool live,
                                         const Place<T, D, kStyle> &place, const T *weight, float eps,
                                         const Angles<T, D> &ang) {
  using A = Angles<T, D>;
  constexpr int kBatch = 4;
  if (from >= to) return;
  int h = from * A::kGroups + group;
  src += h * in;
  dst += h * out;
  in *= A::kGroups;
  out *= A::kGroups;
  uint4 raw[kBatch];
  auto load = [&](int j) {
    const T *row = src;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (live && j + i < to && h + i * A::kGroups < heads) raw[i] = place.load(row);
      row += in;
    }
    src = row;
  };
  load(from);
  Factors<T, D, kStyle> f;
  if (!kCopy) f.set(ang, place, weight);
  for (int j = from; j < to; j += kBatch) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!kCopy) raw[i] = f.apply(raw[i], place, eps);
      if (live && j + i < to && h + i * A::kGroups < heads) place.store(dst, raw[i]);
      dst += out;
    }
    h += kBatch * A::kGroups;
    if (j + kBatch < to) load(j + kBatch);
  }
}

// The sequence of a row that is appended, and its position, from row to row of a warp's
// stretch.
struct Cells {
  int seq = -1, end = -1, len = 0;  // the last row's sequence, where it ends, its length
  int pos;
  __device__ __forceinline__ void at(const RopeArgs &a, int t, int lane) {
    if (t >= end) {
      seq = seq_of_row(a.batch, t, lane);
      if (seq >= 0) {
        end = min(a.batch.q_starts[seq + 1], a.tokens);
        len = max(a.batch.kv_lengths[seq], 0);
      }
    }
    // tokens up to the sequence's end count back from its length
    pos = seq >= 0 ? len - (end - t) : 0;
  }
  __device__ __forceinline__ bool live() const { return seq >= 0; }
  // row of head 0 in the cache; -1: none
  __device__ __forceinline__ long long cell(const RopeArgs &a) const {
    return seq >= 0 ? paged_cell(a.batch, seq, pos, 0, a.Hkv) : -1;
  }
  __device__ __forceinline__ int angle(const RopeArgs &a, int t) const {
    return append_angle(a, t, seq, pos);
  }
};

template <typename T, int D, int kStyle, bool kAppend>
__global__ void __launch_bounds__(kThreads, kFwdCtas) rope_fwd_kernel(const RopeArgs a, int warps) {
  using A = Angles<T, D>;
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % A::kLanes, group = lane / A::kLanes;
  const Place<T, D, kStyle> place(col, a.rotary);
  const int rq = (a.H + A::kGroups - 1) / A::kGroups, rk = (a.Hkv + A::kGroups - 1) / A::kGroups;
  const int rounds = rq + (kAppend ? 2 : 1) * rk;
  const int w = blockIdx.x * kWarps + warp;
  griddep_wait();
  if (w >= warps) return;
  A ang;
  ang.frequencies(a.inv_freq, place.freq, place.on, group);
  Stretch stretch(static_cast<long long>(a.tokens) * rounds, w, warps);
  int t, lo, hi;
  Cells cells;
  while (stretch.next(rounds, t, lo, hi)) {
    bool live = true;
    if (kAppend) {
      cells.at(a, t, lane);
      live = cells.live();
      ang.at(cells.angle(a, t), col);
    } else {
      ang.at(a.positions != nullptr ? a.positions[t] : t % a.L, col);
    }
    const int layout = kAppend ? kLayoutBSHD : a.layout;
    const Rows q = rows_of(layout, t, a.H, a.L, D), k = rows_of(layout, t, a.Hkv, a.L, D);
    fwd_rows<T, D, kStyle, false>(static_cast<const T *>(a.q) + q.base, q.step,
                                  static_cast<T *>(a.q_out) + q.base, q.step, a.H, lo,
                                  min(hi, rq), group, live, place,
                                  static_cast<const T *>(a.q_weight), a.eps, ang);
    Rows to = k;
    if (kAppend) {
      const long long cell = cells.cell(a);
      live = cell >= 0;
      to.base = cell * D;
      to.step = a.batch.layout == kLayoutBHSD ? static_cast<long long>(a.batch.page_size) * D : D;
    }
    fwd_rows<T, D, kStyle, false>(static_cast<const T *>(a.k) + k.base, k.step,
                                  static_cast<T *>(a.k_out) + to.base, to.step, a.Hkv,
                                  max(lo - rq, 0), min(hi - rq, rk), group, live, place,
                                  static_cast<const T *>(a.k_weight), a.eps, ang);
    if (kAppend)
      fwd_rows<T, D, kStyle, true>(static_cast<const T *>(a.v) + k.base, k.step,
                                   static_cast<T *>(a.v_out) + to.base, to.step, a.Hkv,
                                   max(lo - rq - rk, 0), hi - rq - rk, group, live, place,
                                   nullptr, 0.f, ang);
  }
}

// Appending where a token has at most kShortRounds rounds of each tensor (8 heads of 64 in
// bf16): all its rows are loaded at once, ahead of the loads that find its sequence, position
// and cell, which only the stores need.
constexpr int kShortRounds = 2;
template <typename T, int D, int kStyle>
__global__ void __launch_bounds__(kThreads, kFwdCtas)
    rope_append_short_kernel(const RopeArgs a, int warps) {
  using A = Angles<T, D>;
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % A::kLanes, group = lane / A::kLanes;
  const Place<T, D, kStyle> place(col, a.rotary);
  const int rq = (a.H + A::kGroups - 1) / A::kGroups, rk = (a.Hkv + A::kGroups - 1) / A::kGroups;
  const int w = blockIdx.x * kWarps + warp;
  griddep_wait();
  if (w >= warps) return;
  A ang;
  ang.frequencies(a.inv_freq, place.freq, place.on, group);
  const int rounds = rq + 2 * rk;
  Stretch stretch(static_cast<long long>(a.tokens) * rounds, w, warps);
  const long long step =
      (a.batch.layout == kLayoutBHSD ? static_cast<long long>(a.batch.page_size) : 1) * D * A::kGroups;
  int t, lo, hi;
  Cells cells;
  while (stretch.next(rounds, t, lo, hi)) {
    const long long q0 = (static_cast<long long>(t) * a.H + group) * D;
    const long long k0 = (static_cast<long long>(t) * a.Hkv + group) * D;
    // which of the rounds are this warp's, and this lane's rows there
    bool mine[3][kShortRounds];
    uint4 raw[3][kShortRounds];
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const T *src = static_cast<const T *>(x == 0 ? a.q : (x == 1 ? a.k : a.v)) + (x == 0 ? q0 : k0);
#pragma unroll
      for (int i = 0; i < kShortRounds; ++i) {
        const int j = (x == 0 ? 0 : (x == 1 ? rq : rq + rk)) + i;
        mine[x][i] = i < (x == 0 ? rq : rk) && j >= lo && j < hi &&
                     group + i * A::kGroups < (x == 0 ? a.H : a.Hkv);
        raw[x][i] = make_uint4(0, 0, 0, 0);
        if (mine[x][i]) raw[x][i] = place.load(src + i * A::kGroups * D);
      }
    }
    cells.at(a, t, lane);
    const long long cell = cells.cell(a);
    ang.at(cells.angle(a, t), col);
    Factors<T, D, kStyle> f;
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      if (x < 2) f.set(ang, place, static_cast<const T *>(x == 0 ? a.q_weight : a.k_weight));
      T *dst = static_cast<T *>(x == 0 ? a.q_out : (x == 1 ? a.k_out : a.v_out)) +
               (x == 0 ? q0 : cell * D + group * (step / A::kGroups));
      const bool live = x == 0 ? cells.live() : cell >= 0;
#pragma unroll
      for (int i = 0; i < kShortRounds; ++i) {
        if (i >= (x == 0 ? rq : rk)) break;
        if (x < 2) raw[x][i] = f.apply(raw[x][i], place, a.eps);
        if (mine[x][i] && live) place.store(dst + (x == 0 ? i * A::kGroups * D : i * step), raw[x][i]);
      }
    }
  }
}

// Where a token's rows lie in q and k, from token to token without a division.
struct Token {
  long long q, k, step;  // element offsets of heads 0, step per head
  int l;
  __device__ __forceinline__ Token(const RopeArgs &a, int t, int d) {
    const Rows rq = rows_of(a.layout, t, a.H, a.L, d), rk = rows_of(a.layout, t, a.Hkv, a.L, d);
    q = rq.base;
    k = rk.base;
    step = rq.step;
    l = a.layout == kLayoutBSHD ? 0 : t % a.L;
  }
  __device__ __forceinline__ void next(const RopeArgs &a, int d) {
    if (a.layout == kLayoutBSHD) {
      q += static_cast<long long>(a.H) * d;
      k += static_cast<long long>(a.Hkv) * d;
    } else {
      q += d;
      k += d;
      if (++l == a.L) {  // past the other heads' rows, to the next sequence's first
        l = 0;
        q += (a.H - 1) * step;
        k += (a.Hkv - 1) * step;
      }
    }
  }
};

// The backward's rows on their way in.  A warp copies the rounds of its stretch
// kSlots - 1 rounds before it works on them, into its own slots of shared memory: every
// lane reads back what it copied itself, so nothing is waited for but the copies, and
// they go on across heads and tokens (60 -> 47 us on 2 x 4096 tokens of 32 + 8 heads, d
// 128, against loads a round ahead into registers).  A copy goes to the slot whose round
// was worked on last, never to the one being read.  6 slots: 47 us as well; 3 CTAs per
// SM, with fewer registers: 69.
template <typename T, int D, int kStyle>
struct Ahead {
  static constexpr int G = Angles<T, D>::kGroups;
  const RopeArgs &a;
  const Place<T, D, kStyle> &place;
  Token token;
  const T *g, *x;       // this lane's row of the next round: dy, x (null: not needed)
  int left;             // rounds still to be copied
  int group, h, heads;  // its head, of how many
  int more;             // rounds of this token's tensor still to be copied
  bool of_q;
  int slot;
  uint32_t at;  // this lane's 32 bytes of slot 0: dy's two pieces, x's two pieces
  __device__ __forceinline__ Ahead(const RopeArgs &args, const Place<T, D, kStyle> &pl, int t, int r,
                                   int rounds, int rq, int rk, int grp, uint32_t base)
      : a(args), place(pl), token(args, t, D), left(rounds), group(grp), slot(0), at(base) {
    of_q = r < rq;
    if (left > 0) tensor(of_q ? r : r - rq, of_q ? rq : rk);
  }
  // round `from` of `rounds` comes next
  __device__ __forceinline__ void tensor(int from, int rounds) {
    h = from * G + group;
    heads = of_q ? a.H : a.Hkv;
    more = rounds - from;
    const long long first = (of_q ? token.q : token.k) + h * token.step + place.lo;
    g = static_cast<const T *>(of_q ? a.dq_out : a.dk_out) + first;
    const void *rows = of_q ? a.q : a.k;
    x = (of_q ? a.q_weight : a.k_weight) != nullptr ? static_cast<const T *>(rows) + first : nullptr;
  }
  // starts the next round's copies (an absent row's places are zeroed)
  __device__ __forceinline__ void start(int rq, int rk) {
    if (left > 0) {
      const bool is = h < heads;
      const uint32_t dst = at + slot * kSlotBytes;
      copy8(dst, g, is);
      copy8(dst + 256, g + place.apart, is);
      if (x != nullptr) {
        copy8(dst + 512, x, is);
        copy8(dst + 768, x + place.apart, is);
        x += G * token.step;
      }
      g += G * token.step;
      h += G;
      slot = slot + 1 == kSlots ? 0 : slot + 1;
      if (--left > 0 && --more == 0) {
        of_q = !of_q;
        if (of_q ? rq == 0 : rk == 0) {  // one tensor alone
          of_q = !of_q;
          token.next(a, D);
        } else if (of_q) {
          token.next(a, D);
        }
        tensor(0, of_q ? rq : rk);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

// Gradients of rounds [from, to) of one tensor; this lane's share of the weight's
// gradient is added to dw.
template <typename T, int D, int kStyle>
__device__ __forceinline__ void bwd_rows(Ahead<T, D, kStyle> &ahead, int rq, int rk, int &slot, T *dx,
                                         long long step, int heads, int from, int to,
                                         const Place<T, D, kStyle> &place, bool normed, uint4 weight,
                                         float eps, const Angles<T, D> &ang,
                                         uint64_t (&da)[Place<T, D, kStyle>::kTwos],
                                         uint64_t (&db)[Place<T, D, kStyle>::kTwos]) {
  using P = Place<T, D, kStyle>;
  using A = Angles<T, D>;
  constexpr int kTwos = P::kTwos;
  if (from >= to) return;
  uint64_t wa[kTwos], wb[kTwos];
  P::unpack(weight, wa, wb);
  int h = from * A::kGroups + ahead.group;
  dx += h * step;
  step *= A::kGroups;
#pragma unroll 1
  for (int j = from; j < to; ++j) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
    const uint32_t src = ahead.at + slot * kSlotBytes;
    const uint4 raw_g = lds8x2(src), raw_x = normed ? lds8x2(src + 512) : make_uint4(0, 0, 0, 0);
    slot = slot + 1 == kSlots ? 0 : slot + 1;
    ahead.start(rq, rk);
    const bool is = h < heads;
    uint64_t ga[kTwos], gb[kTwos];
    P::unpack(raw_g, ga, gb);
    if (place.on) {
#pragma unroll
      for (int e = 0; e < kTwos; ++e) {
        const uint64_t a = ga[e], b = gb[e];
        ga[e] = fma2(b, ang.s[e], mul2(a, ang.c[e]));
        gb[e] = fma2(mul2(a, both(-1.f)), ang.s[e], mul2(b, ang.c[e]));
      }
    }
    if (normed) {
      uint64_t xa[kTwos], xb[kTwos], va[kTwos], vb[kTwos];
      P::unpack(raw_x, xa, xb);
      uint64_t sq2 = 0ull, dot2 = 0ull;
#pragma unroll
      for (int e = 0; e < kTwos; ++e) {
        va[e] = mul2(ga[e], wa[e]);
        vb[e] = mul2(gb[e], wb[e]);
        sq2 = fma2(xb[e], xb[e], fma2(xa[e], xa[e], sq2));
        dot2 = fma2(vb[e], xb[e], fma2(va[e], xa[e], dot2));
      }
      const float sq = row_sum<A::kLanes>(sum2(sq2)), dot = row_sum<A::kLanes>(sum2(dot2));
      const float inv = rsqrtf(sq * (1.f / D) + eps);
      // minus inv^2 times the mean of (w g) x
      const uint64_t m = both(-(dot * (1.f / D)) * inv * inv), i2 = both(inv);
      const uint64_t add = both(is ? inv : 0.f);  // an absent row adds nothing (its inv may be infinite)
#pragma unroll
      for (int e = 0; e < kTwos; ++e) {
        da[e] = fma2(ga[e], mul2(xa[e], add), da[e]);
        db[e] = fma2(gb[e], mul2(xb[e], add), db[e]);
        ga[e] = mul2(i2, fma2(xa[e], m, va[e]));
        gb[e] = mul2(i2, fma2(xb[e], m, vb[e]));
      }
    }
    if (is) place.store(dx, P::pack(ga, gb));
    dx += step;
    h += A::kGroups;
  }
}

template <typename T, int D, int kStyle>
__global__ void __launch_bounds__(kThreads, kBwdCtas) rope_bwd_kernel(const RopeArgs a, int warps) {
  using A = Angles<T, D>;
  using P = Place<T, D, kStyle>;
  __shared__ __align__(16) unsigned char ring[kWarps * kSlots * kSlotBytes];
  float (*sums)[D] = reinterpret_cast<float (*)[D]>(ring);  // when the rows are done
  static_assert(sizeof(float) * kWarps * A::kGroups * D <= sizeof(ring), "the sums fit");
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % A::kLanes, group = lane / A::kLanes;
  const Place<T, D, kStyle> place(col, a.rotary);
  const int rq = (a.H + A::kGroups - 1) / A::kGroups, rk = (a.Hkv + A::kGroups - 1) / A::kGroups;
  const int w = blockIdx.x * kWarps + warp;
  uint64_t qa[P::kTwos], qb[P::kTwos], ka[P::kTwos], kb[P::kTwos];  // the weights' gradients
#pragma unroll
  for (int e = 0; e < P::kTwos; ++e) qa[e] = qb[e] = ka[e] = kb[e] = 0ull;
  // (a warp past the last has an empty stretch: it still joins the sums)
  Stretch stretch(static_cast<long long>(a.tokens) * (rq + rk), min(w, warps - 1), warps);
  if (w >= warps) stretch.at = stretch.end;
  griddep_wait();
  const long long first = stretch.at / (rq + rk);
  Token token(a, static_cast<int>(first), D);
  Ahead<T, D, kStyle> ahead(a, place, static_cast<int>(first),
                            static_cast<int>(stretch.at - first * (rq + rk)),
                            static_cast<int>(stretch.end - stretch.at), rq, rk, group,
                            smem_addr(ring) + warp * (kSlots * kSlotBytes) + lane * 8);
#pragma unroll 1
  for (int i = 0; i < kSlots - 1; ++i) ahead.start(rq, rk);
  auto position = [&](int t) { return a.positions != nullptr ? a.positions[t] : t % a.L; };
  int pos = stretch.at < stretch.end ? position(static_cast<int>(first)) : 0;
  const bool q_normed = a.q_weight != nullptr, k_normed = a.k_weight != nullptr;
  uint4 qw = make_uint4(0, 0, 0, 0), kw = qw;
  if (q_normed) qw = place.load(static_cast<const T *>(a.q_weight));
  if (k_normed) kw = place.load(static_cast<const T *>(a.k_weight));
  A ang;
  ang.frequencies(a.inv_freq, place.freq, place.on, group);
  int t, lo, hi, slot = 0;
  while (stretch.next(rq + rk, t, lo, hi)) {
    const int now = pos;
    if (stretch.at < stretch.end) pos = position(t + 1);
    ang.at(now, col);
    bwd_rows<T, D, kStyle>(ahead, rq, rk, slot, static_cast<T *>(a.q_out) + token.q, token.step, a.H,
                           lo, min(hi, rq), place, q_normed, qw, a.eps, ang, qa, qb);
    bwd_rows<T, D, kStyle>(ahead, rq, rk, slot, static_cast<T *>(a.k_out) + token.k, token.step,
                           a.Hkv, max(lo - rq, 0), hi - rq, place, k_normed, kw, a.eps, ang, ka, kb);
    token.next(a, D);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  // this CTA's sums over its row groups, in a fixed order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which == 0 ? a.q_weight : a.k_weight) == nullptr) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < P::kTwos; ++e) {
      float *row = sums[warp * A::kGroups + group];
      float x, y;
      f2_unpack(which == 0 ? qa[e] : ka[e], x, y);
      row[place.element(2 * e, false)] = x;
      row[place.element(2 * e + 1, false)] = y;
      f2_unpack(which == 0 ? qb[e] : kb[e], x, y);
      row[place.element(2 * e, true)] = x;
      row[place.element(2 * e + 1, true)] = y;
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps * A::kGroups; ++k) v += sums[k][threadIdx.x];
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

template <typename T, int D>
int rounds(int heads) {
  constexpr int g = Angles<T, D>::kGroups;
  return (heads + g - 1) / g;
}

// Warps for a number of rounds: the `resident` ones, but no more than leave each two.
int warps_of(long long total, int resident) {
  return static_cast<int>(std::max(std::min<long long>((total + 1) / 2, resident), 1LL));
}

template <typename T, int D, int kStyle>
cudaError_t fwd(const RopeArgs &a, bool append, int num_sms, cudaStream_t stream) {
  const long long total =
      static_cast<long long>(a.tokens) *
      (rounds<T, D>(a.H) + (append ? 2 : 1) * rounds<T, D>(a.Hkv));
  const int warps = warps_of(total, kFwdCtas * kWarps * num_sms);
  const dim3 grid((warps + kWarps - 1) / kWarps);
  if (append && rounds<T, D>(a.H) <= kShortRounds && rounds<T, D>(a.Hkv) <= kShortRounds)
    return launch(rope_append_short_kernel<T, D, kStyle>, grid, kThreads, stream, a, warps);
  return append ? launch(rope_fwd_kernel<T, D, kStyle, true>, grid, kThreads, stream, a, warps)
                : launch(rope_fwd_kernel<T, D, kStyle, false>, grid, kThreads, stream, a, warps);
}

template <typename T, int D, int kStyle>
cudaError_t bwd(const RopeArgs &a, int num_sms, cudaStream_t stream) {
  const long long total =
      static_cast<long long>(a.tokens) * (rounds<T, D>(a.H) + rounds<T, D>(a.Hkv));
  const int warps =
      warps_of(total, std::min(kBwdCtas * num_sms, kRopeBwdMaxCtas) * kWarps);
  const int grid = total > 0 ? (warps + kWarps - 1) / kWarps : 0;
  cudaError_t e = cudaSuccess;
  if (grid > 0) e = launch(rope_bwd_kernel<T, D, kStyle>, dim3(grid), kThreads, stream, a, warps);
  if (e == cudaSuccess && (a.dq_weight != nullptr || a.dk_weight != nullptr))
    e = launch(rope_dweight_kernel, dim3(D / 32, 2), kSumWarps * 32, stream,
               static_cast<const float *>(a.partial), grid, D, a.dq_weight, a.dk_weight);
  return e;
}

template <typename T, int D, int kStyle>
cudaError_t rope_style(const RopeArgs &a, int mode, int num_sms, cudaStream_t stream) {
  return mode < 2 ? fwd<T, D, kStyle>(a, mode == 1, num_sms, stream)
                  : bwd<T, D, kStyle>(a, num_sms, stream);
}

template <typename T, int D>
cudaError_t rope(const RopeArgs &a, int mode, int num_sms, cudaStream_t stream) {
  if (a.style == kRopeInterleaved) return rope_style<T, D, kInterleaved>(a, mode, num_sms, stream);
  return a.rotary == D ? rope_style<T, D, kWholeHalves>(a, mode, num_sms, stream)
                       : rope_style<T, D, kHalves>(a, mode, num_sms, stream);
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

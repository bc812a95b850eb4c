// Entry points of include/mha_paged.h: argument validation, kernel choice and
// launch on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/mha_paged.h"
#include "buffers.cuh"
#include "common.cuh"
#include "host.cuh"
#include "paged.cuh"

namespace mha {
namespace {

// tokens of the row operators, and a token's rows: their warps step through 32-bit numbers
constexpr long long kMaxTokens = 0x7fffffffLL - (1 << 20);
bool rows_fit(long long tokens, int H, int H_kv, int d) {
  return tokens <= kMaxTokens && H + 2LL * H_kv <= kMaxTokens && fits({tokens, H, d}) &&
         fits({tokens, H_kv, d});
}

// Checks shared by every operator here.
int check_common(int d, int layout, int dtype) {
  if (d <= 0) return MHA_ERR_INVALID_ARGUMENT;
  if (layout != kLayoutBHSD && layout != kLayoutBSHD) return MHA_ERR_INVALID_ARGUMENT;
  if (dtype != MHA_DTYPE_F32 && dtype != MHA_DTYPE_BF16) return MHA_ERR_INVALID_ARGUMENT;
  return d == 64 || d == 128 ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

int check_rope(int d, int rotary_dim, int style, float eps) {
  if (rotary_dim < 0 || rotary_dim > d) return MHA_ERR_INVALID_ARGUMENT;
  if (style != MHA_ROPE_HALVES && style != MHA_ROPE_INTERLEAVED) return MHA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(eps) || eps < 0.f) return MHA_ERR_INVALID_ARGUMENT;
  return rotary_dim % 16 == 0 ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

// Checks of a ragged batch and its cache; fills `b`.
int check_batch(const int32_t *q_starts, const int32_t *kv_lengths, const int32_t *block_table,
                int B, int T, int num_pages, int page_size, int max_pages, int layout,
                PagedBatch *b) {
  if (B < 0 || T < 0 || num_pages < 0 || max_pages < 0) return MHA_ERR_INVALID_ARGUMENT;
  if (page_size <= 0 || (page_size & (page_size - 1)) != 0) return MHA_ERR_INVALID_ARGUMENT;
  if (page_size < 16) return MHA_ERR_UNSUPPORTED;
  b->q_starts = q_starts;
  b->kv_lengths = kv_lengths;
  b->block_table = block_table;
  b->B = B;
  b->T = T;
  b->num_pages = num_pages;
  b->page_size = page_size;
  b->page_shift = 0;
  while ((1 << b->page_shift) < page_size) ++b->page_shift;
  b->max_pages = max_pages;
  b->layout = layout;
  return MHA_OK;
}

// ---- attention over the cache -------------------------------------------------
// Expected query rows per key/value head up to which the few-query kernel is taken.
// Measured at 16 rows, few / many: one token of 16 heads over 1, 8 sequences of 1000-8000
// keys, d 128: 15.8 / 21.7 us; of 64 over 4, 16 such sequences: 36.7 / 46.6; 4 tokens of 32
// heads over 8, 8 of 1000-4000: 27.0 / 30.6, 32 sequences of 500-2000: 41.4 / 47.1, d 64 36.3 /
// 35.0; 256 of 200-600, d 128: 125.8 / 126.4 (12 rows: 129.3 / 126.2).  8 rows, 16 x 2 tokens of
// 32 heads over 8, 4000 keys, d 128: 51.5 / 62.7.  A few-query kernel of 32 rows (with the
// merges that both had before), 64 sequences of 1000-4000: 101 / 84 us, 128 of 300-900: 160 / 87.
constexpr int kFewRows = 16;

enum PagedPath { kNone = 0, kSimt = 1, kFew = 2, kMany = 3 };

// Units of work of a kernel (PagedProblem): heads, tokens, and its CTAs at most.
struct Units {
  int hpu, hblocks, tb, rows, ctas;
  PagedSplit split;
};

int paged_path(int B, int T, int H, int H_kv, int d, int max_q, int dtype) {
  if (B < 0 || T < 0 || H < 0 || max_q < 1) return -MHA_ERR_INVALID_ARGUMENT;
  if (H_kv <= 0 ? H > 0 || H_kv < 0 : H % H_kv != 0) return -MHA_ERR_INVALID_ARGUMENT;
  const int st = check_common(d, kLayoutBHSD, dtype);
  if (st != MHA_OK) return -st;
  // row numbers and tensor-map extents are 32-bit
  if (static_cast<long long>(T) * H > 0x7fffffffLL || static_cast<long long>(B) * H > 0x7fffffffLL)
    return -MHA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0 || H == 0) return kNone;
  if (dtype == MHA_DTYPE_F32) return kSimt;
  return static_cast<long long>(H / H_kv) * max_q <= kFewRows ? kFew : kMany;
}

// `rows`: of a tile; 0: as many as the kernel takes.
Units units_of(int path, int group, int max_q, int rows = 0) {
  Units u;
  if (rows == 0) rows = path == kMany ? 128 : 16;
  u.hpu = std::min(group, rows);
  u.hblocks = (group + u.hpu - 1) / u.hpu;
  u.tb = path == kMany ? 2 * (rows / u.hpu) : std::min(rows / u.hpu, max_q);
  u.rows = u.hpu * u.tb;
  u.ctas = path == kMany || rows > 16 ? kPagedManyMaxCtas : kPagedMaxCtas;
  u.split = path == kMany ? kSplitMany : (path == kFew ? kSplitFew : kSplitSimt);
  return u;
}

// Trees of drafted tokens have many rows to a sequence, and where the sequences are few or
// short most SMs would have nothing to do: units of fewer rows read the keys again, from
// L2, but a row's softmax no longer waits for 15 others.  `path` and the answer: the rows of
// a unit, 0 where the usual units are as good; `path` becomes the few-query kernel where
// that is faster than the many-query one.  How much work there is is known on the device alone:
// here it is what the table has room for, so short sequences in wide tables count as long ones
// (16 tokens over 300 keys, 8 heads, d 64, with room for 320: 8.9 us, 4096: 11.0, 8192: 13.0,
// 16384 and more: 14.2; the fp32 trees of 5-13 tokens over 90-700 keys, room for 736: 14.4, 2048
// and more: 16.4).
//
// Measured, usual units / these, by units x tiles of the longest sequence that the table
// has room for (T4, T8: with 4 and 8 rows).  bf16, d 64, 16 tokens of 8 heads: T4 = 96 12.1
// / 9.0 us, 384 14.9 / 12.9; T8 = 752 18.6 / 15.6; T4 = 1536 13.9 / 14.7; 8 tokens of 8
// heads over 2 (many-query): T4 = 752 17.5 / 13.6, 768 11.6 / 10.4.  d
// 128, 8 tokens of 32 heads over 8 (many-query): T4 = 192 12.4 / 9.5; T8 = 384 18.9 / 14.5,
// 1536 20.2 / 23.4; 16 of 16 heads: T8 = 384 16.7 / 14.5, 1504 20.4 / 21.8.  fp32, 4 / 8 /
// 16 rows, sequences that fill their tables: d 64, 13 tokens of 8 heads over 2: T4 = 312 13.4 /
// 13.6 / 13.8 us, 624 16.4 / 16.5 / 17.9, T8 = 1008 25.3 / 23.7 / 23.4; 16 tokens of 8 heads:
// T4 = 96 10.3 / 11.7 / 11.5, 768 18.0 / 16.7 / 18.8, T8 = 768 25.5 / 22.4 / 21.9.  d 128,
// 16 tokens of 8 heads: T4 = 96 11.3 / 16.1 / 15.1, T8 = 192 19.7 / 17.4 / 21.0, 384 28.4 /
// 24.1 / 22.1.  Ragged ones, of an eighth to all of it: d 64, 4 tokens of 16 heads over 4: T4 =
// 1024 12.4 / 14.4 / 18.3; 5-13 of 8 over 2: T4 = 1248 15.2 / 15.9 / 17.5, T8 = 1344 19.2 /
// 17.4 / 19.7; 6-16 of 8: T8 = 1024 18.6 / 16.6 / 18.5, 1536 22.6 / 21.4 / 20.8; d 128, T4 =
// 384 13.7 / 14.6 / 20.2, T8 = 672 22.8 / 20.5 / 21.6, 1344 31.3 / 28.2 / 27.0.
//
// Large fp32 trees at d 128 take 32 rows to a unit, where that makes for fewer units of the
// mean tree.  16 / 32 rows, by T32: 8 of 32 tokens of 8 heads, 1000 keys, 512: 59.0 / 50.3 us;
// 64 of 500 keys, 2560: 196 / 151; 13 tokens of 8 heads over 2, 256: 33.5 / 28.7, ragged 384
// 27.3 / 28.9; 32 tokens, ragged, 192: 26.7 / 28.1; 8-20 tokens of 8 heads (one unit either
// way), 4096: 123 / 157.  One CTA of them fits an SM, so there are as few slots for their sums
// as the many-query kernel has; with twice as many, the workspace, which is that of the usual
// units, had no room for the 27 or 30 rows of groups of 6, 9 and 10 heads: 16 of 64 tokens of 12
// heads over 2, 1000 keys: 328 / 213 us; of 18: 638 / 343; 2 of 150 tokens of 10 heads over 1,
// 4000 keys: 351 / 194.
int tree_rows(int *path, int B, int T, int H_kv, int group, int max_q, int d, int dtype,
              long long keys, int sms) {
  const long long tiles = (keys + kPagedTile - 1) / kPagedTile;
  const bool f32 = dtype == MHA_DTYPE_F32;
  const long long ctas = (d == 64 ? 2LL : 1LL) * sms;
  const auto work = [&](const Units &u) {
    const long long blocks =
        std::min<long long>(T, static_cast<long long>(B) * ((max_q - 1LL) / u.tb + 1));
    return blocks * H_kv * u.hblocks * tiles;
  };
  const Units usual = units_of(*path, group, max_q);
  for (const int rows : {4, 8}) {
    const Units u = units_of(kFew, group, max_q, rows);
    if (u.rows >= usual.rows) continue;
    const long long most =
        rows == 4 ? (d == 128 ? 2 : (f32 ? 3 : 4)) : (d == 128 && !f32 ? 3 : 4);
    if (work(u) <= most * ctas) {
      if (*path == kMany) *path = kFew;
      return rows;
    }
  }
  if (f32 && d == 128) {
    const Units u = units_of(*path, group, max_q, 32);
    const long long mean = (T - 1LL) / B + 1;  // tokens of a sequence
    const auto units = [&](const Units &x) { return ((mean - 1) / x.tb + 1) * x.hblocks; };
    if (3 * units(u) <= 2 * units(usual) && 2 * work(u) > 3 * ctas) return 32;
  }
  return 0;
}

size_t meta_bytes(const Units &u) {
  return round_up(sizeof(int32_t) * kPagedMeta * static_cast<size_t>(u.ctas));
}
size_t workspace_bytes_of(const Units &u, int d) {
  return meta_bytes(u) + round_up(sizeof(float) * 2 * static_cast<size_t>(u.ctas) *
                                  paged_slot_floats(u.rows, d));
}

}  // namespace
}  // namespace mha

using namespace mha;

extern "C" int mha_qk_norm_rope_fwd(const void *q, const void *k, void *q_out, void *k_out,
                                    const void *q_weight, const void *k_weight,
                                    const int32_t *positions, const float *inv_freq, int B, int H,
                                    int H_kv, int L, int d, int rotary_dim, int layout, int style,
                                    float eps, int dtype, void *stream) {
  if (B < 0 || H < 0 || H_kv < 0 || L < 0) return MHA_ERR_INVALID_ARGUMENT;
  int st = check_common(d, layout, dtype);
  if (st == MHA_OK) st = check_rope(d, rotary_dim, style, eps);
  if (st != MHA_OK) return st;
  const long long tokens = static_cast<long long>(B) * L;
  if (!rows_fit(tokens, H, H_kv, d)) return MHA_ERR_UNSUPPORTED;
  if (tokens == 0 || (H == 0 && H_kv == 0)) return MHA_OK;
  const size_t e = elem_size(dtype);
  const size_t nq = static_cast<size_t>(tokens) * H * d * e;
  const size_t nk = static_cast<size_t>(tokens) * H_kv * d * e;
  const Buffer outs[2] = {{q_out, nq, 16}, {k_out, nk, 16}};
  const Buffer ins[6] = {{q, nq, 16},
                         {k, nk, 16},
                         {q_weight, q_weight != nullptr && nq > 0 ? d * e : 0, 16},
                         {k_weight, k_weight != nullptr && nk > 0 ? d * e : 0, 16},
                         {positions, positions != nullptr ? tokens * sizeof(int32_t) : 0, 4},
                         {inv_freq, rotary_dim / 2 * sizeof(float), 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {0, 1})) return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.H = H;
  a.Hkv = H_kv;
  a.L = L;
  a.tokens = static_cast<int>(tokens);
  a.rotary = rotary_dim;
  a.layout = layout;
  a.style = style;
  a.eps = eps;
  return launch_rope_fwd(a, d, dtype, false, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? MHA_OK
             : MHA_ERR_CUDA;
}

extern "C" size_t mha_qk_norm_rope_bwd_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  return round_up(sizeof(float) * 2 * static_cast<size_t>(kRopeBwdMaxCtas) * d);
}

extern "C" int mha_qk_norm_rope_bwd(const void *q, const void *k, const void *dq_out,
                                    const void *dk_out, void *dq, void *dk, float *dq_weight,
                                    float *dk_weight, const void *q_weight, const void *k_weight,
                                    const int32_t *positions, const float *inv_freq, int B, int H,
                                    int H_kv, int L, int d, int rotary_dim, int layout, int style,
                                    float eps, int dtype, void *workspace, size_t workspace_bytes,
                                    void *stream) {
  if (B < 0 || H < 0 || H_kv < 0 || L < 0) return MHA_ERR_INVALID_ARGUMENT;
  int st = check_common(d, layout, dtype);
  if (st == MHA_OK) st = check_rope(d, rotary_dim, style, eps);
  if (st != MHA_OK) return st;
  const long long tokens = static_cast<long long>(B) * L;
  if (!rows_fit(tokens, H, H_kv, d)) return MHA_ERR_UNSUPPORTED;
  if ((q_weight == nullptr) != (dq_weight == nullptr) ||
      (k_weight == nullptr) != (dk_weight == nullptr))
    return MHA_ERR_INVALID_ARGUMENT;
  const bool weights = q_weight != nullptr || k_weight != nullptr;
  const size_t e = elem_size(dtype);
  const size_t nq = static_cast<size_t>(tokens) * H * d * e;
  const size_t nk = static_cast<size_t>(tokens) * H_kv * d * e;
  const size_t nw = weights ? mha_qk_norm_rope_bwd_workspace_size(d) : 0;
  if (nw > 0 && workspace_bytes < nw) return MHA_ERR_INVALID_ARGUMENT;
  const Buffer outs[5] = {{dq, nq, 16},
                          {dk, nk, 16},
                          {dq_weight, dq_weight != nullptr ? d * sizeof(float) : 0, 16},
                          {dk_weight, dk_weight != nullptr ? d * sizeof(float) : 0, 16},
                          {workspace, nw, kAlign}};
  const Buffer ins[8] = {
      {dq_out, nq, 16},
      {dk_out, nk, 16},
      {q, q_weight != nullptr ? nq : 0, 16},
      {k, k_weight != nullptr ? nk : 0, 16},
      {q_weight, q_weight != nullptr ? d * e : 0, 16},
      {k_weight, k_weight != nullptr ? d * e : 0, 16},
      {positions, positions != nullptr ? tokens * sizeof(int32_t) : 0, 4},
      {inv_freq, tokens > 0 ? rotary_dim / 2 * sizeof(float) : 0, 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {0, 1, -1, -1, -1}))
    return MHA_ERR_INVALID_ARGUMENT;
  if (nq + nk == 0 && !weights) return MHA_OK;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  RopeArgs a{};
  a.q = q;
  a.k = k;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.q_out = dq;
  a.k_out = dk;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  a.partial = static_cast<float *>(workspace);
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.H = H;
  a.Hkv = H_kv;
  a.L = L;
  a.tokens = nq + nk > 0 ? static_cast<int>(tokens) : 0;
  a.rotary = rotary_dim;
  a.layout = layout;
  a.style = style;
  a.eps = eps;
  return launch_rope_bwd(a, d, dtype, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MHA_OK
             : MHA_ERR_CUDA;
}

// mha_paged_append and mha_paged_append_at: `at` says whether the angles' positions are
// given.
static int append(const void *q, const void *k, const void *v, void *q_out, void *k_cache,
                  void *v_cache, const void *q_weight, const void *k_weight, const float *inv_freq,
                  bool at, const int32_t *positions, const int32_t *q_starts,
                  const int32_t *kv_lengths, const int32_t *block_table, int B, int T, int H,
                  int H_kv, int d, int num_pages, int page_size, int max_pages, int rotary_dim,
                  int layout, int style, float eps, int dtype, void *stream) {
  if (H < 0 || H_kv < 0) return MHA_ERR_INVALID_ARGUMENT;
  if (H_kv == 0 ? H > 0 : H % H_kv != 0) return MHA_ERR_INVALID_ARGUMENT;
  int st = check_common(d, layout, dtype);
  if (st == MHA_OK) st = check_rope(d, rotary_dim, style, eps);
  RopeArgs a{};
  if (st == MHA_OK)
    st = check_batch(q_starts, kv_lengths, block_table, B, T, num_pages, page_size, max_pages,
                     layout, &a.batch);
  if (st != MHA_OK) return st;
  if (!rows_fit(T, H, H_kv, d) || !fits({num_pages, page_size, H_kv, d}) ||
      !fits({B, max_pages}))
    return MHA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0 || H_kv == 0) return MHA_OK;
  const size_t e = elem_size(dtype);
  const size_t nq = static_cast<size_t>(T) * H * d * e;
  const size_t nk = static_cast<size_t>(T) * H_kv * d * e;
  const size_t nc = static_cast<size_t>(num_pages) * page_size * H_kv * d * e;
  const Buffer outs[3] = {{q_out, nq, 16}, {k_cache, nc, 16}, {v_cache, nc, 16}};
  const Buffer ins[10] = {
      {q, nq, 16},
      {k, nk, 16},
      {v, nk, 16},
      {q_weight, q_weight != nullptr && nq > 0 ? d * e : 0, 16},
      {k_weight, k_weight != nullptr ? d * e : 0, 16},
      {inv_freq, rotary_dim / 2 * sizeof(float), 4},
      {positions, at ? sizeof(int32_t) * static_cast<size_t>(T) : 0, 4},
      {q_starts, sizeof(int32_t) * (static_cast<size_t>(B) + 1), 4},
      {kv_lengths, sizeof(int32_t) * static_cast<size_t>(B), 4},
      {block_table, sizeof(int32_t) * static_cast<size_t>(B) * max_pages, 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {0, -1, -1}))
    return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.k_out = k_cache;
  a.v_out = v_cache;
  // (a weight of no queries has not been looked at, and the kernels form every weight's factors)
  a.q_weight = nq > 0 ? q_weight : nullptr;
  a.k_weight = k_weight;
  a.inv_freq = inv_freq;
  a.positions = at ? positions : nullptr;
  a.H = H;
  a.Hkv = H_kv;
  a.L = T;
  a.tokens = T;
  a.rotary = rotary_dim;
  a.layout = kLayoutBSHD;
  a.style = style;
  a.eps = eps;
  return launch_rope_fwd(a, d, dtype, true, sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? MHA_OK
             : MHA_ERR_CUDA;
}

extern "C" int mha_paged_append(const void *q, const void *k, const void *v, void *q_out,
                                void *k_cache, void *v_cache, const void *q_weight,
                                const void *k_weight, const float *inv_freq,
                                const int32_t *q_starts, const int32_t *kv_lengths,
                                const int32_t *block_table, int B, int T, int H, int H_kv, int d,
                                int num_pages, int page_size, int max_pages, int rotary_dim,
                                int layout, int style, float eps, int dtype, void *stream) {
  return append(q, k, v, q_out, k_cache, v_cache, q_weight, k_weight, inv_freq, false, nullptr,
                q_starts, kv_lengths, block_table, B, T, H, H_kv, d, num_pages, page_size,
                max_pages, rotary_dim, layout, style, eps, dtype, stream);
}

extern "C" int mha_paged_append_at(const void *q, const void *k, const void *v, void *q_out,
                                   void *k_cache, void *v_cache, const void *q_weight,
                                   const void *k_weight, const float *inv_freq,
                                   const int32_t *positions, const int32_t *q_starts,
                                   const int32_t *kv_lengths, const int32_t *block_table, int B,
                                   int T, int H, int H_kv, int d, int num_pages, int page_size,
                                   int max_pages, int rotary_dim, int layout, int style, float eps,
                                   int dtype, void *stream) {
  return append(q, k, v, q_out, k_cache, v_cache, q_weight, k_weight, inv_freq, true, positions,
                q_starts, kv_lengths, block_table, B, T, H, H_kv, d, num_pages, page_size,
                max_pages, rotary_dim, layout, style, eps, dtype, stream);
}

extern "C" int mha_paged_path(int B, int T, int H, int H_kv, int d, int max_q, int page_size,
                              int dtype) {
  PagedBatch b;
  const int st = check_batch(nullptr, nullptr, nullptr, B, T, 0, page_size, 0, kLayoutBHSD, &b);
  if (st != MHA_OK) return -st;
  return paged_path(B, T, H, H_kv, d, max_q, dtype);
}

extern "C" size_t mha_paged_workspace_size(int B, int T, int H, int H_kv, int d, int max_q,
                                           int dtype) {
  const int path = paged_path(B, T, H, H_kv, d, max_q, dtype);
  if (path <= kNone) return 0;
  return workspace_bytes_of(units_of(path, H / H_kv, max_q), d);
}

// The CTAs that a call's shapes have work for, at most `grid`: what no sequence can
// need is not launched (one token over 300 keys of 8 heads: 24 CTAs, not 304).
static int launched_ctas(const PagedProblem &p, int grid) {
  const long long blocks = std::min<long long>(p.batch.T, p.batch.B + p.batch.T / p.tb);
  const long long units = blocks * p.Hkv * p.hblocks;
  if (units >= grid) return grid;
  const long long keys = static_cast<long long>(p.batch.max_pages) << p.batch.page_shift;
  const long long tiles = (keys + kPagedTile - 1) / kPagedTile;
  const long long total = units * (p.split.unit_cost + kTileCost / 2 + tiles * kTileCost);
  return static_cast<int>(
      std::max(1LL, std::min<long long>(grid, paged_ctas(total, units, p.split.stretches))));
}

// mha_paged_fwd and mha_paged_tree_fwd: `of_tree` says whether tokens see one another as
// the tree says.
static int attend(const void *q, const void *k_cache, const void *v_cache, void *out, bool of_tree,
                  const uint32_t *tree, int tree_words, const int32_t *q_starts,
                  const int32_t *kv_lengths, const int32_t *block_table, int B, int T, int H,
                  int H_kv, int d, int max_q, int num_pages, int page_size, int max_pages,
                  int layout, int mask_kind, float scale, int dtype, void *workspace,
                  size_t workspace_bytes, void *stream_) {
  int st = check_common(d, layout, dtype);
  PagedProblem p{};
  if (st == MHA_OK)
    st = check_batch(q_starts, kv_lengths, block_table, B, T, num_pages, page_size, max_pages,
                     layout, &p.batch);
  if (st != MHA_OK) return st;
  int path = paged_path(B, T, H, H_kv, d, max_q, dtype);
  if (path < 0) return -path;
  if (mask_kind != MHA_MASK_NONE && mask_kind != MHA_MASK_CAUSAL_TAIL)
    return MHA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || (of_tree && tree_words < 1)) return MHA_ERR_INVALID_ARGUMENT;
  if (!fits({num_pages, page_size, H_kv, d}) || !fits({B, max_pages}) || !fits({T, tree_words}))
    return MHA_ERR_UNSUPPORTED;
  // the kernels count keys, and a few tiles past them, in 32 bits
  if ((static_cast<long long>(max_pages) << p.batch.page_shift) > (1LL << 31) - 1024)
    return MHA_ERR_UNSUPPORTED;
  if (path == kNone) return MHA_OK;
  Units u = units_of(path, H / H_kv, max_q);
  const size_t e = elem_size(dtype);
  const size_t nq = static_cast<size_t>(T) * H * d * e;
  const size_t nc = static_cast<size_t>(num_pages) * page_size * H_kv * d * e;
  const size_t nw = workspace_bytes_of(u, d);
  if (workspace_bytes < nw) return MHA_ERR_INVALID_ARGUMENT;
  const Buffer outs[2] = {{out, nq, 16}, {workspace, nw, kAlign}};
  const size_t nt = of_tree ? sizeof(uint32_t) * static_cast<size_t>(T) * tree_words : 0;
  const Buffer ins[7] = {{q, nq, 16},
                         {k_cache, nc, 16},
                         {v_cache, nc, 16},
                         {tree, nt, 4},
                         {q_starts, sizeof(int32_t) * (static_cast<size_t>(B) + 1), 4},
                         {kv_lengths, sizeof(int32_t) * static_cast<size_t>(B), 4},
                         {block_table, sizeof(int32_t) * static_cast<size_t>(B) * max_pages, 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {-1, -1}))
    return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
  if (of_tree) {
    int small_path = path;
    const int rows =
        tree_rows(&small_path, B, T, H_kv, H / H_kv, max_q, d, dtype,
                  static_cast<long long>(max_pages) << p.batch.page_shift, sms);
    const Units small = units_of(small_path, H / H_kv, max_q, rows);
    if (rows > 0 && workspace_bytes_of(small, d) <= nw) {
      path = small_path;
      u = small;
    }
  }
  p.H = H;
  p.Hkv = H_kv;
  p.group = H / H_kv;
  p.hpu = u.hpu;
  p.hblocks = u.hblocks;
  p.tb = u.tb;
  p.rows = u.rows;
  p.causal = mask_kind == MHA_MASK_CAUSAL_TAIL;
  p.scale_log2 = scale * kLog2e;
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.out = out;
  p.meta = static_cast<int32_t *>(workspace);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + meta_bytes(u));
  p.status = status_ptr();
  if (p.status == nullptr) return MHA_ERR_CUDA;
  p.wait_ns = wait_limit_ns();
  p.stall = wait_stall();
  if (of_tree) {
    p.tree = tree;
    p.tree_words = tree_words;
  }
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  p.split = u.split;
  int grid = launched_ctas(p, u.ctas);
  cudaError_t err = cudaSuccess;
  if (path == kSimt) {
    grid = std::min(grid, (d == 64 ? 2 : 1) * sms);  // CTAs that run at a time
    err = launch_paged_simt(p, d, grid, stream);
  } else {
    CUtensorMap qm, km, vm;
    const int box = std::min(page_size, kPagedTile);
    // a cache without pages is never read: any valid map will do
    const bool none = num_pages == 0;
    const void *kb = none ? q : k_cache, *vb = none ? q : v_cache;
    const int pages = none ? 1 : num_pages;
    if (!make_map(&qm, q, d, T, H, 1, kLayoutBSHD, path == kMany ? u.tb / 2 : u.tb, u.hpu) ||
        !make_map(&km, kb, d, page_size, H_kv, pages, layout, box, 1) ||
        !make_map(&vm, vb, d, page_size, H_kv, pages, layout, box, 1))
      return MHA_ERR_CUDA;
    if (path == kMany) {
      grid = std::min(grid, sms);
      err = launch_paged_many(qm, km, vm, p, d, grid, stream);
    } else {
      err = launch_paged_few(qm, km, vm, p, d, grid, sms, stream);
    }
  }
  // a unit is cut only when both parts have min_part tiles: not where the block
  // table has no room for them
  const long long most = static_cast<long long>(max_pages) * page_size;
  if (err == cudaSuccess && most > (2 * u.split.min_part - 1) * kPagedTile)
    err = launch_paged_merge(p, d, dtype, path == kMany, grid, sms, stream);
  return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

extern "C" int mha_paged_fwd(const void *q, const void *k_cache, const void *v_cache, void *out,
                             const int32_t *q_starts, const int32_t *kv_lengths,
                             const int32_t *block_table, int B, int T, int H, int H_kv, int d,
                             int max_q, int num_pages, int page_size, int max_pages, int layout,
                             int mask_kind, float scale, int dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
  return attend(q, k_cache, v_cache, out, false, nullptr, 0, q_starts, kv_lengths, block_table, B,
                T, H, H_kv, d, max_q, num_pages, page_size, max_pages, layout, mask_kind, scale,
                dtype, workspace, workspace_bytes, stream);
}

extern "C" int mha_paged_tree_fwd(const void *q, const void *k_cache, const void *v_cache,
                                  void *out, const int32_t *tree_mask, const int32_t *q_starts,
                                  const int32_t *kv_lengths, const int32_t *block_table, int B,
                                  int T, int H, int H_kv, int d, int max_q, int num_pages,
                                  int page_size, int max_pages, int tree_words, int layout,
                                  float scale, int dtype, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  return attend(q, k_cache, v_cache, out, true, reinterpret_cast<const uint32_t *>(tree_mask),
                tree_words, q_starts, kv_lengths, block_table, B, T, H, H_kv, d, max_q, num_pages,
                page_size, max_pages, layout, MHA_MASK_NONE, scale, dtype, workspace,
                workspace_bytes, stream);
}

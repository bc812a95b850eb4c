// Entry points of include/mha_paged.h: argument validation, kernel choice and
// launch on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/mha_paged.h"
#include "common.cuh"
#include "host.cuh"
#include "paged.cuh"

namespace mha {
namespace {

constexpr size_t kAlign = 256;
size_t round_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// One argument's memory: where, how much, the alignment it needs.
struct Buffer {
  const void *p;
  size_t n;
  size_t align;
};

// Whether every buffer with a size is there and aligned.
template <size_t N>
bool present(const Buffer (&bufs)[N]) {
  for (const Buffer &b : bufs)
    if (b.n > 0 && (b.p == nullptr || reinterpret_cast<uintptr_t>(b.p) % b.align != 0)) return false;
  return true;
}

// Whether an output shares memory with an input or another output; output i may
// be input in_place[i] itself (same address).
template <size_t N, size_t M>
bool clash(const Buffer (&outs)[N], const Buffer (&ins)[M], const int (&in_place)[N]) {
  for (size_t o = 0; o < N; ++o) {
    for (size_t i = 0; i < M; ++i) {
      if (static_cast<int>(i) == in_place[o] && outs[o].p == ins[i].p) continue;
      if (overlaps(outs[o].p, outs[o].n, ins[i].p, ins[i].n)) return true;
    }
    for (size_t o2 = o + 1; o2 < N; ++o2)
      if (overlaps(outs[o].p, outs[o].n, outs[o2].p, outs[o2].n)) return true;
  }
  return false;
}

// Whether a product of counts (>= 0) stays below 2^56: sizes in bytes then fit.
bool fits(std::initializer_list<long long> counts) {
  long long n = 1;
  for (const long long c : counts) {
    if (c != 0 && n > (1LL << 56) / c) return false;
    n *= c;
  }
  return true;
}

// tokens of the row operators, and a token's rows: their warps step through 32-bit numbers
constexpr long long kMaxTokens = 0x7fffffffLL - (1 << 20);
bool rows_fit(long long tokens, int H, int H_kv, int d) {
  return tokens <= kMaxTokens && H + 2LL * H_kv <= kMaxTokens && fits({tokens, H, d}) &&
         fits({tokens, H_kv, d});
}

size_t elem_size(int dtype) { return dtype == MHA_DTYPE_F32 ? 4 : 2; }

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

// SMs of the current device; 0 on failure
int current_sms() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? sm_count(dev) : 0;
}

// ---- attention over the cache -------------------------------------------------
// Expected query rows per key/value head up to which the few-query kernel is taken.
// Measured at 16 rows, few / many: one token of 16 heads over 1, 8 sequences of 1000-8000
// keys, d 128: 17 / 32 us; of 64 over 4, 16 such sequences: 38 / 49; 4 tokens of 32 heads
// over 8, 32 sequences of 500-2000, d 128: 44 / 50.  Units short beside their number go the
// other way: the same 32 sequences at d 64: 41 / 36; 256 of 200-600, d 128: 144 / 129 (12
// rows: 141 / 129).  8 rows, 16 x 2 tokens of 32 heads over 8, 4000 keys, d 128: 52 / 66.
// A few-query kernel of 32 rows, 64 sequences of 1000-4000: 101 / 84 us, 128 of 300-900:
// 160 / 87.
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

Units units_of(int path, int group, int max_q) {
  Units u;
  const int rows = path == kMany ? 128 : 16;  // of a tile
  u.hpu = std::min(group, rows);
  u.hblocks = (group + u.hpu - 1) / u.hpu;
  u.tb = path == kMany ? 2 * (rows / u.hpu) : std::min(rows / u.hpu, max_q);
  u.rows = u.hpu * u.tb;
  u.ctas = path == kMany ? kPagedManyMaxCtas : kPagedMaxCtas;
  u.split = path == kMany ? kSplitMany : (path == kFew ? kSplitFew : kSplitSimt);
  return u;
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

extern "C" int mha_paged_append(const void *q, const void *k, const void *v, void *q_out,
                                void *k_cache, void *v_cache, const void *q_weight,
                                const void *k_weight, const float *inv_freq,
                                const int32_t *q_starts, const int32_t *kv_lengths,
                                const int32_t *block_table, int B, int T, int H, int H_kv, int d,
                                int num_pages, int page_size, int max_pages, int rotary_dim,
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
  const Buffer ins[9] = {
      {q, nq, 16},
      {k, nk, 16},
      {v, nk, 16},
      {q_weight, q_weight != nullptr && nq > 0 ? d * e : 0, 16},
      {k_weight, k_weight != nullptr ? d * e : 0, 16},
      {inv_freq, rotary_dim / 2 * sizeof(float), 4},
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
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.inv_freq = inv_freq;
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

extern "C" int mha_paged_fwd(const void *q, const void *k_cache, const void *v_cache, void *out,
                             const int32_t *q_starts, const int32_t *kv_lengths,
                             const int32_t *block_table, int B, int T, int H, int H_kv, int d,
                             int max_q, int num_pages, int page_size, int max_pages, int layout,
                             int mask_kind, float scale, int dtype, void *workspace,
                             size_t workspace_bytes, void *stream_) {
  int st = check_common(d, layout, dtype);
  PagedProblem p{};
  if (st == MHA_OK)
    st = check_batch(q_starts, kv_lengths, block_table, B, T, num_pages, page_size, max_pages,
                     layout, &p.batch);
  if (st != MHA_OK) return st;
  const int path = paged_path(B, T, H, H_kv, d, max_q, dtype);
  if (path < 0) return -path;
  if (mask_kind != MHA_MASK_NONE && mask_kind != MHA_MASK_CAUSAL_TAIL)
    return MHA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale)) return MHA_ERR_INVALID_ARGUMENT;
  if (!fits({num_pages, page_size, H_kv, d}) || !fits({B, max_pages})) return MHA_ERR_UNSUPPORTED;
  // the kernels count keys, and a few tiles past them, in 32 bits
  if ((static_cast<long long>(max_pages) << p.batch.page_shift) > (1LL << 31) - 1024)
    return MHA_ERR_UNSUPPORTED;
  if (path == kNone) return MHA_OK;
  const Units u = units_of(path, H / H_kv, max_q);
  const size_t e = elem_size(dtype);
  const size_t nq = static_cast<size_t>(T) * H * d * e;
  const size_t nc = static_cast<size_t>(num_pages) * page_size * H_kv * d * e;
  const size_t nw = workspace_bytes_of(u, d);
  if (workspace_bytes < nw) return MHA_ERR_INVALID_ARGUMENT;
  const Buffer outs[2] = {{out, nq, 16}, {workspace, nw, kAlign}};
  const Buffer ins[6] = {{q, nq, 16},
                         {k_cache, nc, 16},
                         {v_cache, nc, 16},
                         {q_starts, sizeof(int32_t) * (static_cast<size_t>(B) + 1), 4},
                         {kv_lengths, sizeof(int32_t) * static_cast<size_t>(B), 4},
                         {block_table, sizeof(int32_t) * static_cast<size_t>(B) * max_pages, 4}};
  if (!present(outs) || !present(ins) || clash(outs, ins, {-1, -1}))
    return MHA_ERR_INVALID_ARGUMENT;
  const int sms = current_sms();
  if (sms <= 0) return MHA_ERR_CUDA;
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
    err = launch_paged_merge(p, d, dtype, path == kMany, grid, stream);
  return err == cudaSuccess ? MHA_OK : MHA_ERR_CUDA;
}

// Definitions shared by the operators of include/mha_paged.h: the ragged batch
// and the paged cache as the kernels see them, and the split of attention work
// over CTAs.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "common.cuh"

// The logic that turns lengths and tables into work is plain integer code and
// also compiles for the host, where its tests run.
#define MHA_HD __host__ __device__ __forceinline__

namespace mha {

// ---- norm and rotation of head rows (qk_rope.cu) ---------------------------
constexpr int kRopeHalves = 0;
constexpr int kRopeInterleaved = 1;

// The ragged batch and its cache (include/mha_paged.h, "Ragged batches").
struct PagedBatch {
  const int32_t *q_starts, *kv_lengths, *block_table;
  int B, T;
  int num_pages, page_size, page_shift, max_pages;  // page_size = 1 << page_shift
  int layout;                                       // of the cache
};

struct RopeArgs {
  const void *q, *k, *v;  // v only when appending
  void *q_out, *k_out, *v_out;  // appending: k_out, v_out are the caches
  const void *q_weight, *k_weight;  // nullptr: that tensor is not normed
  const float *inv_freq;
  const int32_t *positions;  // [B, L], or when appending [tokens]; nullptr: from the place
  int H, Hkv, L;             // not appending: token t = (t / L, t % L)
  int tokens;                // B * L, or the batch's T
  int rotary, layout, style;
  float eps;
  PagedBatch batch;  // appending
  // backward: q, k the forward's inputs, dq_out, dk_out the incoming gradients
  const void *dq_out, *dk_out;
  float *partial;  // [CTAs, 2, d] sums of the weights' gradients
  float *dq_weight, *dk_weight;
};

// The position whose angles appended row t takes, of sequence `seq` (-1: none) and at `pos` of
// it: the given one (drafted trees: it is not the cell's), unread where the row has no sequence.
MHA_HD int append_angle(const RopeArgs &a, int t, int seq, int pos) {
  return a.positions != nullptr && seq >= 0 ? a.positions[t] : pos;
}

// CTAs of the backward kernel at most (rows of RopeArgs::partial)
constexpr int kRopeBwdMaxCtas = 1216;

cudaError_t launch_rope_fwd(const RopeArgs &a, int d, int dtype, bool append, int num_sms,
                            cudaStream_t stream);
cudaError_t launch_rope_bwd(const RopeArgs &a, int d, int dtype, int num_sms, cudaStream_t stream);

// ---- attention over the cache ----------------------------------------------
constexpr int kPagedTile = 128;     // keys per tile: the unit that work is split by
constexpr int kPagedMaxCtas = 608;      // CTAs that may hold partial sums, at most 16 rows per unit
constexpr int kPagedManyMaxCtas = 192;  // ... 256 rows per unit, or 32 in fp32: one CTA to an SM

// What a visible score counts as at least.  A score that is not seen is -infinity, and a
// visible one of -infinity this, so that a row with nothing to attend to (maximum
// -infinity, written as +0.0) is told from one all of whose scores are -infinity (maximum
// kLowestScore: 0 / 0, NaN); next to any other score both weigh 0.
constexpr float kLowestScore = -3.402823466e38f;

constexpr int kTileCost = 256;  // 2^8: shifts below
static_assert(kTileCost == 1 << 8, "tile cost");

// How a kernel's work is split, in key tiles.
struct PagedSplit {
  int unit_cost;    // a unit's own work (queries, first and last tile, output), in 1/256 tile
  int min_part;     // tiles of a part at least
  int stretches;    // CTAs that 2^16 tiles of work are worth: fewer tiles, no CTA of their own
  int half_tile;    // a tile of a unit that has at most half its tokens, in 1/256 tile
  int half_per;     // 2^16 / half_tile
};
// Units cost the tensor-core kernels the time of 1.5 tiles besides their keys (the
// many-query one, with 3 and cuts from 3 tiles on: chunks 84 us, not 80), the fp32
// kernel's one.  The many-query kernel's units with tokens for one warpgroup only take
// 0.8 of the time per tile.  A tile of the fp32 kernel takes about 2 us, so there every
// tile may have a CTA of its own (44 -> 26 us on 8 sequences of 90 to 700 keys, 5 tokens
// of 8 heads).
constexpr PagedSplit kSplitSimt{kTileCost, 1, 65536, kTileCost, 256};
constexpr PagedSplit kSplitFew{kTileCost * 3 / 2, 2, 65536 / 3, kTileCost, 256};
constexpr PagedSplit kSplitMany{kTileCost * 3 / 2, 2, 65536 / 3, 215, 305};

// A unit of attention work: `tb` consecutive new tokens of one sequence times
// `hpu` query heads of one key/value head's group.  Row r of a unit is head
// r / tb of its heads, token r % tb of its tokens.
struct PagedProblem {
  PagedBatch batch;
  int H, Hkv, group;  // group = H / Hkv
  int hpu, hblocks;   // query heads per unit; units that cover a group's heads
  int tb;             // tokens per unit
  int causal;
  PagedSplit split;
  float scale_log2;  // scale * log2(e)
  const void *q, *k, *v;
  void *out;
  // Sums of units whose keys several CTAs share: slot s of CTA c holds `rows`
  // rows of d fp32 (unnormalised output) and, behind them all, (max, sum) pairs
  float *part;
  int32_t *meta;  // [CTAs][kPagedMeta]
  int rows;       // rows of a slot
  int *status;
  uint64_t wait_ns;
  int stall;  // test hook: kStall* bits (common.cuh)
  // Trees of drafted tokens (nullptr: none; then `causal` says what a token sees): bit m
  // of row t's `tree_words` words is set when token t sees new token m of its sequence.
  // What lies before the new tokens every one of them sees.
  const uint32_t *tree;
  int tree_words;
};

// meta words of a CTA: which parts of split units it holds.  Slot 0 holds a part
// that continues a unit begun by the CTA before, slot 1 the first part of a
// unit that the CTAs behind it continue.
constexpr int kPagedMeta = 8;
constexpr int kMetaFlags = 0;  // kPart* bits
// unit of slot 0: first row of out, its tokens, first query head, query heads
constexpr int kMetaRow = 1, kMetaTokens = 2, kMetaHead = 3, kMetaHeads = 4;
constexpr int kPartContinues = 1;  // slot 0 is used
constexpr int kPartEnds = 2;       // ... and holds the unit's last keys
constexpr int kPartBegins = 4;     // slot 1 is used

// Sequence b of a batch: its first row, new tokens, cached length (what the
// block table can hold of it) and the position of its first new token.
struct PagedSeq {
  int q0, n, len, base;
};

MHA_HD PagedSeq paged_seq(const PagedBatch &p, int b) {
  PagedSeq s;
  const int a = p.q_starts[b], e = p.q_starts[b + 1], l = p.kv_lengths[b];
  s.q0 = min(max(a, 0), p.T);
  s.n = min(max(e, s.q0), p.T) - s.q0;
  const int full = max(l, 0);
  const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
  s.len = static_cast<int>(min(static_cast<long long>(full), cap));
  s.base = full - s.n;
  return s;
}

// Keys that tokens [i0, i1) of a sequence may read, at most.
MHA_HD int paged_kv_end(const PagedSeq &s, int i1, int causal) {
  if (!causal) return s.len;
  return max(min(s.base + i1, s.len), 0);
}

// ---- trees of drafted tokens -----------------------------------------------
// Word i of a token's row; 0 outside it.
MHA_HD uint32_t tree_word(const uint32_t *row, int words, int i) {
  return static_cast<unsigned>(i) < static_cast<unsigned>(words) ? row[i] : 0u;
}
// Which of 32 positions a token sees, the first `from` positions behind its sequence's
// first new token (negative: before it): lo and hi are words from >> 5 and the one behind.
MHA_HD uint32_t tree_window(uint32_t lo, uint32_t hi, int from) {
  const int s = from & 31;
#ifdef __CUDA_ARCH__
  uint32_t see = __funnelshift_r(lo, hi, s);
#else
  uint32_t see = s == 0 ? lo : (lo >> s) | (hi << (32 - s));
#endif
  if (from < 0) see |= from <= -32 ? 0xffffffffu : (1u << -from) - 1u;
  return see;
}

// ---- the split of the units' keys over CTAs --------------------------------
// Units are laid on a line, each as long as its work (in 1/256 of a key tile):
// head block by head block, for each all sequences, for each its token blocks.
// CTA c of G takes the stretch [c X / G, (c + 1) X / G) of the line, X its length;
// a unit's keys are cut where a stretch ends inside it, unless that leaves a part
// of under `min_part` tiles.  G is at most the grid, and no larger than leaves every
// CTA 2^16 / `stretches` tiles or, if that is more, one unit each.
//
// Heads come first because every head's piece of the line is alike: with G a
// multiple of the head blocks, the CTAs of different heads read the same positions
// at about the same time, and in the [page, position, head, d] layout those lie
// side by side in memory (66 -> 58 us on 256 sequences of 128 to 1024 keys, 8
// heads, d 64).

// tiles of a unit (of at most half its tokens: `half`) before offset x (> 0) of its
// piece of the line
MHA_HD int paged_cut(const PagedSplit &sp, bool half, long long x, int nt) {
  if (x <= 0) return 0;
  const long long t = ((x - sp.unit_cost) * (half ? sp.half_per : 256) + 32768) >> 16;
  if (t < sp.min_part) return 0;
  if (t > nt - sp.min_part) return nt;
  return static_cast<int>(t);
}

// A CTA's place on the line: where its stretch begins and ends, and its first unit.
struct PagedSpan {
  long long lo, hi;  // the stretch
  long long at;      // where the first unit begins
  int hb;            // head block of the first unit
  int b;             // its sequence
  int u;             // its token block
  int ctas;          // G
};

// A quotient for a place to start from: a division that rounds is a call.
MHA_HD float paged_about(float a, float b) {
#ifdef __CUDA_ARCH__
  return __fdividef(a, b);
#else
  return a / b;
#endif
}

// CTAs that a line of length `total` with `units` units has work for.
MHA_HD long long paged_ctas(long long total, long long units, int stretches) {
  const long long by_work = (total >> 8) * stretches >> 16;  // kTileCost is 2^8
  const long long most = by_work > units ? by_work : units;
  // a stretch is longer than a tile, so that no CTA between a unit's first and last
  // part is without one (paged_merge_kernel takes them as neighbours)
  const long long cap = (total >> 8) * 31 / 32;
  return most < cap ? most : cap;
}

// The stretch of CTA `cta` of `grid` on a line of length `total` with `units` units.
MHA_HD PagedSpan paged_stretch(long long total, long long units, int cta, int grid,
                               int stretches) {
  PagedSpan sp;
  const long long most = paged_ctas(total, units, stretches);
  sp.ctas = static_cast<int>(most < 1 ? 1 : (most < grid ? most : grid));
  // equal stretches, a little short (the last CTA takes what is left, some millionths):
  // an approximate quotient, for a 64-bit division is a hundred instructions
  const long long each = static_cast<long long>(
      paged_about(static_cast<float>(total), static_cast<float>(sp.ctas)) * 0.999999f);
  sp.lo = cta < sp.ctas ? each * cta : total;
  sp.hi = cta + 1 < sp.ctas ? each * (cta + 1) : total;
  sp.at = total;
  sp.hb = sp.b = sp.u = 0;
  return sp;
}

// token blocks of a sequence: its units of one head block
MHA_HD int paged_blocks(const PagedProblem &p, const PagedSeq &s) { return (s.n + p.tb - 1) / p.tb; }
// Length on the line of unit u of a sequence: exact in tiles when the sequence has
// one token block; else linear in its keys (half a tile for the last, ragged one),
// so that sums over units have a closed form.
MHA_HD int paged_blocks_end(const PagedProblem &p, const PagedSeq &s, int u) {
  const long long i1 = static_cast<long long>(u + 1) * p.tb;
  return i1 < s.n ? static_cast<int>(i1) : s.n;
}
MHA_HD bool paged_half(const PagedProblem &p, const PagedSeq &s, int u) {
  return 2 * (paged_blocks_end(p, s, u) - u * p.tb) <= p.tb;
}
MHA_HD long long paged_unit_cost(const PagedProblem &p, const PagedSeq &s, int blocks, int u) {
  const long long keys = paged_kv_end(s, paged_blocks_end(p, s, u), p.causal);
  const int tile = paged_half(p, s, u) ? p.split.half_tile : kTileCost;
  if (blocks == 1) return p.split.unit_cost + (keys + kPagedTile - 1) / kPagedTile * tile;
  return p.split.unit_cost + kTileCost / 2 + keys * tile / kPagedTile;
}
// Length of the units before u (0 <= u <= blocks) of a sequence.
MHA_HD long long paged_cost_before(const PagedProblem &p, const PagedSeq &s, int blocks, int u) {
  if (u <= 0) return 0;
  const long long last = u == blocks ? paged_unit_cost(p, s, blocks, blocks - 1) : 0;
  const int full = u == blocks ? blocks - 1 : u;  // units before the last
  if (full == 0) return last;
  const long long fixed = p.split.unit_cost + kTileCost / 2, per_key = kTileCost / kPagedTile;
  if (!p.causal) return full * (fixed + per_key * s.len) + last;
  // units before the last see base + (v + 1) tb keys, held to [0, len]
  const unsigned tb = static_cast<unsigned>(p.tb);
  int lo = s.base < 0 ? static_cast<int>((0u - static_cast<unsigned>(s.base)) / tb) : 0;
  if (lo > full) lo = full;  // units that see nothing
  // ... and from `hi` on, all of len
  const unsigned room = s.len > s.base
                            ? static_cast<unsigned>(s.len) - static_cast<unsigned>(s.base) - 1u
                            : 0u;
  int hi = s.len > s.base && room / tb < static_cast<unsigned>(full) ? static_cast<int>(room / tb)
           : s.len > s.base                                          ? full
                                                                     : 0;
  if (hi < lo) hi = lo;
  const long long some = hi - lo;
  const long long keys = some * s.base + ((some * (hi + lo + 1)) >> 1) * p.tb +
                         static_cast<long long>(full - hi) * s.len;
  return full * fixed + per_key * keys + last;
}

// The unit of a sequence whose piece of the line holds offset x, and the length before it.
MHA_HD int paged_unit_at(const PagedProblem &p, const PagedSeq &s, int blocks, long long x,
                         long long &before) {
  int lo = 0, hi = blocks;
  before = 0;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const long long c = paged_cost_before(p, s, blocks, mid);
    if (c <= x) {
      lo = mid;
      before = c;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// The span of CTA `cta` of `grid`; all threads of the block call it (kThreads of
// them), `scratch` holds 40 long longs in shared memory, every thread gets the
// answer.  Ends with a __syncthreads.
template <int kThreads>
__device__ PagedSpan paged_span(const PagedProblem &p, int cta, int grid, long long *scratch) {
  constexpr int kWarps = (kThreads + 31) / 32;
  static_assert(kWarps <= 16, "scratch size");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.batch.B + kThreads - 1) / kThreads;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, p.batch.B), b1 = min(b0 + per, p.batch.B);
  long long mine = 0, units = 0;  // of one head block
  for (int b = b0; b < b1; ++b) {
    const PagedSeq s = paged_seq(p.batch, b);
    const long long nu = paged_blocks(p, s);
    units += nu;
    mine += paged_cost_before(p, s, static_cast<int>(nu), static_cast<int>(nu));
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
    units += __shfl_xor_sync(0xffffffffu, units, o);
  }
  if (lane == 31) {
    scratch[warp] = inc;
    scratch[16 + warp] = units;
  }
  __syncthreads();
  long long before = 0, one = 0, all_units = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scratch[w];
    one += scratch[w];
    all_units += scratch[16 + w];
  }
  const int hbs = p.Hkv * p.hblocks;
  PagedSpan sp = paged_stretch(one * hbs, all_units * hbs, cta, grid, p.split.stretches);
  const bool any = sp.lo < one * hbs;
  int hb = hbs;
  if (any) {  // sp.lo / one, from an approximate quotient
    hb = static_cast<int>(paged_about(static_cast<float>(sp.lo), static_cast<float>(one)));
    while (hb > 0 && hb * one > sp.lo) --hb;
    while ((hb + 1) * one <= sp.lo) ++hb;
  }
  const long long at = any ? sp.lo - hb * one : 0, first = before + inc - mine;
  if (any && at >= first && at < first + mine) {  // one thread of the block
    long long s = first;
    for (int b = b0;; ++b) {
      const PagedSeq q = paged_seq(p.batch, b);
      const int nu = paged_blocks(p, q);
      const long long whole = paged_cost_before(p, q, nu, nu);
      if (at < s + whole || b + 1 >= b1) {
        long long before_u;
        scratch[34] = paged_unit_at(p, q, nu, at - s, before_u);
        scratch[32] = s + before_u;
        scratch[33] = b;
        break;
      }
      s += whole;
    }
  }
  __syncthreads();
  sp.hb = hb;
  if (any) {
    sp.at = hb * one + scratch[32];
    sp.b = static_cast<int>(scratch[33]);
    sp.u = static_cast<int>(scratch[34]);
  }
  return sp;
}

// One CTA's share of a unit: tiles [t0, t1) of its nt.
struct PagedPart {
  PagedSeq seq;
  int b;        // sequence
  int kv;       // key/value head
  int h0;       // first query head
  int heads;    // query heads (the last block of a group may have fewer)
  int i0, i1;   // tokens of the sequence
  int kv_end;   // keys that any of its rows may read
  int nt, t0, t1;
};

// Walks the parts of a CTA's span in order.
struct PagedWalk {
  PagedSpan sp;
  PagedSeq seq, ahead;  // sequence b, and the one behind it (read early)
  int hb, b, u, blocks;
  long long at;  // where unit u begins

  MHA_HD void take(const PagedProblem &p, const PagedSeq &q) {
    seq = q;
    blocks = paged_blocks(p, seq);
    ahead = paged_seq(p.batch, b + 1 < p.batch.B ? b + 1 : 0);
  }
  MHA_HD void begin(const PagedProblem &p, const PagedSpan &span) {
    sp = span;
    hb = sp.hb;
    b = sp.b;
    u = sp.u;
    at = sp.hi;
    if (sp.lo < sp.hi) {
      take(p, paged_seq(p.batch, b));
      at = sp.at;
    }
  }
  // The next part; false when the span is done.
  MHA_HD bool next(const PagedProblem &p, PagedPart &part) {
    for (;;) {
      if (at >= sp.hi) return false;
      while (u >= blocks) {
        u = 0;
        if (++b >= p.batch.B) {
          b = 0;
          if (++hb >= p.Hkv * p.hblocks) return false;  // lengths changed meanwhile
        }
        take(p, ahead);
      }
      part.seq = seq;
      part.b = b;
      part.kv = hb / p.hblocks;
      const int hin = (hb - part.kv * p.hblocks) * p.hpu;
      part.h0 = part.kv * p.group + hin;
      part.heads = p.group - hin < p.hpu ? p.group - hin : p.hpu;
      part.i0 = u * p.tb;
      part.i1 = paged_blocks_end(p, seq, u);
      part.kv_end = paged_kv_end(seq, part.i1, p.causal);
      part.nt = (part.kv_end + kPagedTile - 1) / kPagedTile;
      const long long from = at;
      at += paged_unit_cost(p, seq, blocks, u);
      ++u;
      const bool half = 2 * (part.i1 - part.i0) <= p.tb;
      part.t0 = paged_cut(p.split, half, sp.lo - from, part.nt);
      part.t1 = sp.hi < at ? paged_cut(p.split, half, sp.hi - from, part.nt) : part.nt;
      if (part.nt == 0) {  // nothing to attend to: zeros, by the CTA that holds its beginning
        if (from >= sp.lo) return true;
        continue;
      }
      if (part.t1 > part.t0) return true;
    }
  }
};

MHA_HD bool paged_split(const PagedPart &part) {
  return part.t0 > 0 || part.t1 < part.nt;
}
// slot of a split part
MHA_HD int paged_slot(const PagedPart &part) { return part.t0 > 0 ? 0 : 1; }

// One slot: rows x d sums (of the many-query kernel [d / 4][rows][4]), then rows x
// (max, sum); whole 16-byte pieces, because the sums are read and written 16 bytes at a
// time.
MHA_HD size_t paged_slot_floats(int rows, int d) {
  return (static_cast<size_t>(rows) * (d + 2) + 3) / 4 * 4;
}
MHA_HD float *paged_slot_ptr(const PagedProblem &p, int d, int cta, int slot) {
  return p.part + (static_cast<size_t>(cta) * 2 + slot) * paged_slot_floats(p.rows, d);
}

// Number of the cell [page, head, offset] of position pos in the cache, in rows
// of d; -1 when the position lies in no page.
MHA_HD long long paged_cell(const PagedBatch &p, int b, int pos, int head,
                                                int heads) {
  if (pos < 0) return -1;
  const int pi = pos >> p.page_shift;
  if (pi >= p.max_pages) return -1;
  const int id = p.block_table[static_cast<size_t>(b) * p.max_pages + pi];
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages)) return -1;
  const int off = pos & (p.page_size - 1);
  return p.layout == kLayoutBHSD
             ? ((static_cast<long long>(id) * heads + head) << p.page_shift) + off
             : ((static_cast<long long>(id) << p.page_shift) + off) * heads + head;
}

// bf16, at most 16 rows per unit: maps over q (d, T, H, 1) with box (64, tb, hpu, 1)
// and over the caches (d, page_size, H_kv, num_pages) with box
// (64, min(page_size, 128), 1, 1); lowers `grid` to the CTAs it launches
cudaError_t launch_paged_few(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                             const PagedProblem &p, int d, int &grid, int num_sms,
                             cudaStream_t stream);
// bf16, 256 rows per unit: maps over q with box (64, tb / 2, hpu, 1), over the caches
// as above
cudaError_t launch_paged_many(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                              const PagedProblem &p, int d, int grid, cudaStream_t stream);
// fp32, at most 16 rows per unit, of trees at d = 128 32
cudaError_t launch_paged_simt(const PagedProblem &p, int d, int grid, cudaStream_t stream);
// joins the parts of split units; `many`: of launch_paged_many
cudaError_t launch_paged_merge(const PagedProblem &p, int d, int dtype, bool many, int grid,
                               int num_sms, cudaStream_t stream);

}  // namespace mha

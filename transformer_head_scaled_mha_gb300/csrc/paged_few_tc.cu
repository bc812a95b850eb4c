// Attention of a few query rows against a paged key/value cache on the tcgen05
// tensor cores (bf16, d in {64, 128}): steps of single or a few tokens.
//
// A part of work (paged.cuh) is R <= 16 query rows of one key/value head -- its
// group's query heads times a few tokens -- against some 128-key tiles.  Each key
// and value is read once, so the kernel is bound by HBM.  Persistent CTAs take equal
// stretches of all sequences' tiles, cutting a sequence's keys where a stretch ends;
// paged_merge_kernel joins the cut ones.
//
// Measured, with the merge: one token, 64 sequences of 4096-8192 keys, 32 heads over 8,
// d 128: 230-235 us, 6.9 TB/s (1.02 of a copy's rate); 256 sequences of 128-1024 keys, 8
// heads, d 64: 59 us, 5.1 TB/s (0.76; its 2048 short units and the way to a CTA's first
// tile, 7 us); one sequence of 300 keys: 8.2 us, a chain of latencies.  Batches that do
// not fill the GPU for long pay 6 us to the first tile and 4 for the merge: 8 sequences of
// 1000-4000 keys, 32 heads over 8, d 128: 24.6 us, 0.49 of a copy's rate.  From 9 rows on
// the lone softmax warpgroup sets the pace, 16 exponentials and stores per key and thread:
// 32 sequences of 500-2000 keys, 4 tokens of 32 heads over 8, d 64: 36 us, 0.33.  Trees of
// drafted tokens where there is little work come in units of 4 or 8 rows: 16 tokens over 300
// keys, 8 heads, d 64: 8.9 us (12.1 with 16 rows; 14 where the table has room for 16384
// positions); 256 trees of 8 tokens, 128-1024 keys, 8 heads, d 64: 78 us, 0.58 (89 with a
// quotient to every row in every thread).
//
// Scores are computed transposed, keys on the 128 TMEM lanes, so that a thread
// owns a key and the few rows cost a few exponentials per thread:
//
//   S^T = K_j Q^T        tcgen05.mma M=128 keys, N=16 rows, K=d, both K-major
//   softmax              thread k holds key k's score of every row; a row's tile
//                        maximum by shuffles and a 4-warp exchange; the running
//                        maximum moves only when it grows by more than 2^8
//                        (numerator and denominator share it), and O is rescaled
//                        in TMEM when it does; partial row sums per thread
//   P -> smem (bf16)     up to 8 rows as a sum of two bf16, the second in the
//                        product's padding rows; more rows leave none, and are rounded
//                        to one (2^-8 relative): a second product would double the
//                        stores that set the pace there
//   O^T += V_j^T P^T     A = the V tile read MN-major.  d = 64: both 64-key halves
//                        of the tile in one product, M rows 0..63 the first
//                        half's values and 64..127 the second's, B the first
//                        half's P rows then the second's; the two diagonal blocks
//                        of D are partial outputs, summed at the end
//
// Tiles come page by page: a box of min(page, 128) rows per 64 columns of K and V,
// issued by as many lanes of the producer warp at once (page 16, d = 128: 32
// copies of 2 KB per tile).  Pages that hold no key of the part, or are not there,
// are not loaded; their keys are masked and their value rows, like those behind
// the last key, are zeroed in shared memory, because whatever the cache holds
// there (or an earlier tile left) times a weight of 0 need not be 0.
//
// Warp roles (224 threads): warps 0-3 softmax and output, warp 4 producer, which
// also walks the parts and hands their descriptions to the others, warp 5 TMEM
// owner and score-product issuer, warp 6 PV issuer (two issuers because each
// product costs its issuing thread about 70 cycles).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kThreads = 224;
constexpr int kSoftmaxThreads = 128;
constexpr int kBN = kPagedTile;
constexpr int kN = 16;  // query rows per score product
constexpr uint32_t kTmemCols = 128;  // S0 S1 (kN each), O0 O1 (kOCols each)
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kMaxSlots = 3;
constexpr int kDescs = 4;  // part descriptions in flight
constexpr uint32_t kBarSoftmax = 1;

// d = 64: half the ring and two CTAs per SM, whose waits (for a part's first tile,
// its output, a lone softmax warp's latencies) fall into each other's work.
template <int D, int RP>
struct Cfg {
  static constexpr int kCtas = D == 64 ? 2 : 1;  // per SM
  static constexpr int kSlabs = D / 64;
  static constexpr int kBlkBytes = 128 * 128;           // [128 rows x 64] swizzle block
  static constexpr int kTileBytes = kSlabs * kBlkBytes;  // a K or V tile
  static constexpr int kSlotBytes = 2 * kTileBytes;      // ring slot: K tile, V tile
  static constexpr int kSlots = 3;
  static constexpr int kQBlk = kN * 128;  // [kN rows x 64] of Q
  static constexpr int kQBytes = kSlabs * kQBlk;
  // Up to 8 rows the weights go in as two bf16, the rounded weight and what the
  // rounding left (2^-17 relative together), in rows of the product that would
  // otherwise be padding: row r and row r + kLo.
  static constexpr bool kTwo = RP <= 8;
  static constexpr int kLo = D == 64 && RP <= 4 ? 4 : 8;
  static constexpr int kPRows = D == 64 && RP <= 4 ? 8 : kN;  // rows of P per 64-key half
  static constexpr int kPHalf = kPRows * 128;
  static constexpr int kPBytes = 2 * kPHalf;
  static constexpr int kPvN = D == 64 ? 2 * kPRows : kN;
  static constexpr int kPvSteps = D == 64 ? 4 : 8;
  // A's second M block: d = 64, the tile's keys 64..127 (64 rows down);
  // d = 128, value dims 64..127 (the next swizzle block)
  static constexpr uint32_t kVLbo = D == 64 ? 64 * 128 : kBlkBytes;
  static constexpr int kOCols = kPvN;
  static_assert(2 * kN + 2 * kOCols <= static_cast<int>(kTmemCols), "tensor memory");
};

// A part as the other roles need it.
struct Desc {
  int go;           // 0: no more parts
  int tiles;        // to process (0: rows of zeros)
  int key0;         // first key of the first tile
  int kv_end;       // keys from here on are not attended to
  int lim0;         // keys below this are allowed for the first token
  int lim_step;     // ... plus this per token
  int row0;         // first row of q and out
  int tokens, heads, h0;
  int slot;         // of its sums; -1: the part is a whole unit
};

template <int RP>
struct __align__(16) Shared {
  union {
    float4 red[2][RP];      // tile maxima of the four warps, double-buffered by tile
    long long scratch[40];  // before: where the span is found
  };
  float4 lsum[RP];      // row sums of the four warps
  Desc desc[kDescs];
  uint32_t present[kMaxSlots];  // pages of the slot's tile that were loaded
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  uint64_t s_full[2];   // S_t in TMEM
  uint64_t p_full[2];   // P_t in smem, S_t read (softmax threads)
  uint64_t pv_done[2];  // PV_t done, by tile parity
  uint64_t o_free[2];   // the epilogue has read O of a part
  uint64_t never;       // nothing signals it (test hook)
  uint32_t tmem_base;
  int abort_flag;
};

template <int D, int RP>
constexpr size_t smem_bytes() {
  using C = Cfg<D, RP>;
  return 1024 + static_cast<size_t>(C::kSlots) * C::kSlotBytes + 2 * C::kQBytes + 2 * C::kPBytes +
         sizeof(Shared<RP>);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Maxima of R values (R rows, one value of each per lane) over the warp: halves of
// the rows change hands at each step, so R - 1 + log2(32 / R) shuffles serve all
// rows (5 R row by row).  Lane l ends with row l / (32 / R).
template <int R>
__device__ __forceinline__ float rows_max(float (&v)[R], int lane) {
  int bit = 16;
#pragma unroll
  for (int h = R / 2; h > 0; h >>= 1, bit >>= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    }
  }
  for (; bit > 0; bit >>= 1) v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
  return v[0];
}

struct FewMaps {
  CUtensorMap q;     // (d, T, H, 1), box (64, tb, hpu, 1)
  CUtensorMap k, v;  // (d, page_size, H_kv, num_pages), box (64, min(page_size, 128), 1, 1)
};

// Waits for description n and copies it (a whole warp of a reading role); false
// when there are no more parts, or when the wait was given up (then !ok).
template <int RP>
__device__ __forceinline__ bool take_desc(Shared<RP> *sh, int n, Desc &d, uint64_t limit, bool &ok) {
  volatile int *abort_flag = &sh->abort_flag;
  ok = mbar_wait_warp(&sh->desc_full[n % kDescs], (n / kDescs) & 1, abort_flag, limit);
  if (!ok) return false;
  d = sh->desc[n % kDescs];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh->desc_empty[n % kDescs]);
  return d.go != 0;
}

template <int D, int RP, bool kTree>
__global__ void __launch_bounds__(kThreads, Cfg<D, RP>::kCtas)
    paged_few_tc_kernel(const __grid_constant__ FewMaps maps,
                        const __grid_constant__ PagedProblem p) {
  using C = Cfg<D, RP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *ring = smem;                              // kSlots (K tile, V tile)
  uint8_t *qbuf = ring + C::kSlots * C::kSlotBytes;  // 2 Q buffers
  uint8_t *pbuf = qbuf + 2 * C::kQBytes;             // 2 P buffers
  Shared<RP> *sh = reinterpret_cast<Shared<RP> *>(pbuf + 2 * C::kPBytes);
  volatile int *abort_flag = &sh->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.hpu * p.tb;

  // ---- setup -------------------------------------------------------------
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->q_empty[i], 1);
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i], kSoftmaxThreads);
      mbar_init(&sh->pv_done[i], 1);
      mbar_init(&sh->o_free[i], kSoftmaxThreads);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&sh->desc_full[i], 1);
      mbar_init(&sh->desc_empty[i], 6);  // four softmax warps, two issuers
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sh->kv_full[s], 1);
      mbar_init(&sh->kv_empty[s], 1);
    }
    mbar_init(&sh->never, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 5) {
    tmem_alloc(&sh->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  // The next launch may begin only when this CTA has its tensor memory: a CTA of it that
  // allocated first could hold what this one waits for, and itself wait for this launch.
  __syncthreads();
  griddep_launch_dependents();
  griddep_wait();  // lengths, queries and cache come from earlier work
  const PagedSpan span = paged_span<kThreads>(p, blockIdx.x, gridDim.x, sh->scratch);
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  int issued = 0, q_issued = 0;  // producer: K/V and Q loads issued
  uint64_t *last_commit = nullptr;
  uint32_t last_parity = 0;

  if (warp == 4) {
    // ---- producer: walks the parts; per part Q, then (K_j, V_j) ------------
    const PagedBatch &pb = p.batch;
    const int box = min(pb.page_size, kBN);        // rows of a copy
    const int pieces_shift = 7 - min(pb.page_shift, 7);
    const int pieces = 1 << pieces_shift;          // copies per 64 columns of a tile
    const bool loads = lane < 2 * C::kSlabs * pieces;
    const int piece = lane & (pieces - 1);
    const int slab = loads ? (lane >> pieces_shift) % C::kSlabs : 0;
    const int kv = loads ? (lane >> pieces_shift) / C::kSlabs : 0;  // 0: K, 1: V
    const CUtensorMap *map = kv == 0 ? &maps.k : &maps.v;
    const int dst0 = kv * C::kTileBytes + slab * C::kBlkBytes + piece * box * 128;
    PagedWalk walk;
    walk.begin(p, span);
    PagedPart part;
    int n = 0, flags = 0, mrow = 0, mtokens = 0, mhead = 0, mheads = 0;
    bool ok = true;
    for (;;) {
      const bool more = walk.next(p, part);
      const int32_t *table = pb.block_table + static_cast<size_t>(more ? part.b : 0) * pb.max_pages;
      // page of this lane's copy of tile j; -1 when it holds no key or is not there
      auto page_of = [&](int j) -> int {
        const int key = j * kBN + piece * box;
        if (!loads || j >= part.t1 || key >= part.kv_end) return -1;
        const int id = table[key >> pb.page_shift];
        return static_cast<unsigned>(id) < static_cast<unsigned>(pb.num_pages) ? id : -1;
      };
      int id = more ? page_of(part.t0) : -1;
      ok = mbar_wait_warp(&sh->desc_empty[n % kDescs], ((n / kDescs) & 1) ^ 1, abort_flag,
                          p.wait_ns);
      if (!ok) break;
      const bool split = more && paged_split(part);
      if (lane == 0) {
        Desc d;
        d.go = more;
        d.tiles = part.t1 - part.t0;
        d.key0 = part.t0 * kBN;
        d.kv_end = part.kv_end;
        // of a tree: where its tokens begin
        d.lim0 = kTree ? part.seq.base : (p.causal ? part.seq.base + part.i0 + 1 : part.seq.len);
        d.lim_step = p.causal;
        d.row0 = part.seq.q0 + part.i0;
        d.tokens = part.i1 - part.i0;
        d.heads = part.heads;
        d.h0 = part.h0;
        d.slot = split ? paged_slot(part) : -1;
        sh->desc[n % kDescs] = d;
        mbar_arrive(&sh->desc_full[n % kDescs]);
      }
      __syncwarp();
      ++n;
      if (!more) break;
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
      if (part.nt == 0) continue;
      const int qb = q_issued & 1;
      ok = mbar_wait_warp(&sh->q_empty[qb], ((q_issued >> 1) & 1) ^ 1, abort_flag, p.wait_ns);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh->q_full[qb], static_cast<uint32_t>(C::kSlabs * R * 128));
        for (int blk = 0; blk < C::kSlabs; ++blk)
          tma_load_4d(qbuf + qb * C::kQBytes + blk * C::kQBlk, &maps.q, &sh->q_full[qb], blk * 64,
                      part.seq.q0 + part.i0, part.h0, 0);
      }
      ++q_issued;
      for (int j = part.t0; j < part.t1; ++j) {
        const int id_next = page_of(j + 1);
        const int slot = issued % C::kSlots, round = issued / C::kSlots;
        ok = mbar_wait_warp(&sh->kv_empty[slot], (round & 1) ^ 1, abort_flag, p.wait_ns);
        if (!ok) break;
        const uint32_t there = __ballot_sync(0xffffffffu, id >= 0) & ((1u << pieces) - 1);
        if (lane == 0) {
          sh->present[slot] = there;
          mbar_arrive_expect_tx(&sh->kv_full[slot],
                                static_cast<uint32_t>(__popc(there) * box * 128 * 2 * C::kSlabs));
        }
        __syncwarp();
        if (id >= 0)
          tma_load_4d(ring + slot * C::kSlotBytes + dst0, map, &sh->kv_full[slot], slab * 64,
                      (j * kBN + piece * box) & (pb.page_size - 1), part.kv, id);
        ++issued;
        id = id_next;
      }
      if (!ok) break;
    }
    if (lane == 0) {
      int32_t *meta = p.meta + static_cast<size_t>(blockIdx.x) * kPagedMeta;
      meta[kMetaFlags] = flags;
      meta[kMetaRow] = mrow;
      meta[kMetaTokens] = mtokens;
      meta[kMetaHead] = mhead;
      meta[kMetaHeads] = mheads;
    }
  } else if (warp == 5) {
    // ---- score products S_t = K_t Q^T (lane 0 issues; the warp waits) -----
    const uint32_t idesc_s = idesc_bf16_f32(128, kN, 0);
    bool ok = true;
    int t = 0, qi = 0, slot = 0, round = 0;
    Desc d;
    for (int n = 0; ok && take_desc(sh, n, d, p.wait_ns, ok); ++n) {
      if (d.tiles == 0) continue;
      const int qb = qi & 1;
      ok = mbar_wait_warp(&sh->q_full[qb], (qi >> 1) & 1, abort_flag, p.wait_ns);
      for (int j = 0; j < d.tiles && ok; ++j) {
        ok = mbar_wait_warp(&sh->kv_full[slot], round & 1, abort_flag, p.wait_ns);
        // S buffer t % 2 held S_{t-2}: the softmax has read it once P_{t-2} is out
        if (ok && t >= 2)
          ok = mbar_wait_warp(&sh->p_full[t & 1], ((t - 2) >> 1) & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t da0 = smem_desc_sw128(smem_addr(ring + slot * C::kSlotBytes), 16, 1024);
          const uint64_t db0 = smem_desc_sw128(smem_addr(qbuf + qb * C::kQBytes), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ka = (kk >> 2) * C::kBlkBytes + (kk & 3) * 32;
            const uint32_t kb = (kk >> 2) * C::kQBlk + (kk & 3) * 32;
            tc_mma_ss(tmem + (t & 1) * kN, da0 + (ka >> 4), db0 + (kb >> 4), idesc_s,
                      kk > 0 ? 1u : 0u);
          }
          tc_commit(&sh->s_full[t & 1]);
          if (j == d.tiles - 1) tc_commit(&sh->q_empty[qb]);
        }
        __syncwarp();
        last_commit = &sh->s_full[t & 1];
        last_parity = (t >> 1) & 1;
        ++t;
        if (++slot == C::kSlots) {
          slot = 0;
          ++round;
        }
      }
      ++qi;
    }
  } else if (warp == 6) {
    // ---- PV products O (+)= P_t V_t (lane 0 issues; the warp waits) --------
    const uint32_t idesc_o = idesc_bf16_f32_amn(128, C::kPvN, 0);
    // test hook: a wait on a barrier that nothing signals, with copies and score products
    // in flight
    bool ok = (p.stall & kStallPagedFewMma) == 0 ||
              mbar_wait_warp(&sh->never, 0, abort_flag, p.wait_ns);
    int t = 0, oi = 0, slot = 0, round = 0;
    Desc d;
    for (int n = 0; ok && take_desc(sh, n, d, p.wait_ns, ok); ++n) {
      if (d.tiles == 0) continue;
      const uint32_t d_tmem = tmem + 2 * kN + (oi & 1) * C::kOCols;
      for (int j = 0; j < d.tiles && ok; ++j) {
        // P_t written (so S_t, and with it this slot's K and V, had landed)
        ok = mbar_wait_warp(&sh->p_full[t & 1], (t >> 1) & 1, abort_flag, p.wait_ns);
        // the part's first product overwrites O: its epilogue two parts back is done
        if (ok && j == 0)
          ok = mbar_wait_warp(&sh->o_free[oi & 1], ((oi >> 1) & 1) ^ 1, abort_flag, p.wait_ns);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          // A = V^T: 16 key rows per step (8-row groups 1024 B apart)
          const uint64_t da0 = smem_desc_sw128(
              smem_addr(ring + slot * C::kSlotBytes + C::kTileBytes), C::kVLbo, 1024);
          // B = P: 16 keys = 32 bytes of each 128-byte row
          const uint64_t db0 = smem_desc_sw128(smem_addr(pbuf + (t & 1) * C::kPBytes), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < C::kPvSteps; ++kk) {
            // d = 64: the P rows of both halves per step; d = 128: 16 rows, the
            // second 64 keys kPHalf further
            const uint32_t pb = D == 64 ? kk * 32 : (kk >> 2) * C::kPHalf + (kk & 3) * 32;
            tc_mma_ss(d_tmem, da0 + ((kk * 16 * 128) >> 4), db0 + (pb >> 4), idesc_o,
                      (j > 0 || kk > 0) ? 1u : 0u);
          }
          tc_commit(&sh->pv_done[t & 1]);
          tc_commit(&sh->kv_empty[slot]);
        }
        __syncwarp();
        last_commit = &sh->kv_empty[slot];
        last_parity = round & 1;
        ++t;
        if (++slot == C::kSlots) {
          slot = 0;
          ++round;
        }
      }
      ++oi;
    }
  } else {
    // ---- softmax and output: thread k = key k of a tile / TMEM lane k ------
    const int k = threadIdx.x;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    // O^T lanes: d = 128, value dim k; d = 64, value dim k % 64 of the first
    // (warps 0-1) or second (warps 2-3) key half's partial output
    const int o_col = D == 64 && warp >= 2 ? C::kPRows : 0;
    const int vdim = D == 64 ? (k & 63) : k;
    const bool stores = D == 128 || warp < 2;  // threads that write output
    const int box_shift = min(p.batch.page_shift, 7);
    uint16_t *out = static_cast<uint16_t *>(p.out);
    bool ok = true;
    int t = 0, oi = 0, slot = 0, round = 0;
    Desc d;
    for (int n = 0;; ++n) {
      // every softmax warp passes a barrier after its last description, taken or
      // not: a warp that gave up here meets the others at their next one
      if (!take_desc(sh, n, d, p.wait_ns, ok)) {
        (void)named_barrier_and(kBarSoftmax, kSoftmaxThreads, ok);
        break;
      }
      // row r: head r / tb, token r % tb; element vdim of its output
      auto row_at = [&](int h, int i) -> size_t {
        return static_cast<size_t>(d.row0 + i) * p.H + d.h0 + h;
      };
      if (d.tiles == 0) {  // nothing to attend to
        if (stores)
          for (int h = 0; h < d.heads; ++h)
            for (int i = 0; i < d.tokens; ++i) out[row_at(h, i) * D + vdim] = 0;
        continue;
      }
      float m[RP], l[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      int j = 0;
      for (; j < d.tiles; ++j) {
        // Of a tree: tokens that see this thread's key, bit by token.  Their words are
        // loaded before the waits; only a sequence's last tiles need any.
        uint32_t seen = 0xffffffffu;
        if (kTree && d.key0 + j * kBN + kBN > d.lim0) {
          const int m = d.key0 + j * kBN + k - d.lim0;
          if (m >= 0) {
            seen = 0;
            const uint32_t *tree = p.tree + static_cast<size_t>(d.row0) * p.tree_words;
#pragma unroll 4
            for (int tok = 0; tok < d.tokens; ++tok, tree += p.tree_words)
              seen |= ((tree_word(tree, p.tree_words, m >> 5) >> (m & 31)) & 1u) << tok;
          }
        }
        const bool okw =
            mbar_wait_warp(&sh->kv_full[slot], round & 1, abort_flag, p.wait_ns) &&
            mbar_wait_warp(&sh->s_full[t & 1], (t >> 1) & 1, abort_flag, p.wait_ns);
        const int key = d.key0 + j * kBN + k;
        float x[RP];
        if (okw) {
          tc_fence_after();
          uint32_t s[RP];
          tmem_ld_cols(tmem + lane_base + (t & 1) * kN, s);
          const bool there = key < d.kv_end && ((sh->present[slot] >> (k >> box_shift)) & 1);
          const bool all = __all_sync(0xffffffffu, there);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            x[r] = max_nan(__uint_as_float(s[r]) * p.scale_log2, kLowestScore);
            if (RP > 1 && r >= R) x[r] = -INFINITY;  // padding rows of the product
          }
          // a tile that crosses some row's limit, or has keys that are not there
          if (!all || d.key0 + j * kBN + kBN > d.lim0) {
            int tok = 0;
#pragma unroll
            for (int r = 0; r < RP; ++r) {
              const bool sees = kTree ? (seen >> tok) & 1u : key < d.lim0 + tok * d.lim_step;
              if (!there || !sees) x[r] = -INFINITY;
              if (++tok == p.tb) tok = 0;
            }
            if (!there) {  // this key's value row: zeros (chunk order avoids bank conflicts)
              const uint32_t v = smem_addr(ring + slot * C::kSlotBytes + C::kTileBytes) + k * 128;
#pragma unroll
              for (int c = 0; c < 8 * C::kSlabs; ++c)
                st_shared_v4(v + (c >> 3) * C::kBlkBytes + (((c ^ k) & 7) << 4), 0, 0, 0, 0);
            }
          }
          float v[RP];
#pragma unroll
          for (int r = 0; r < RP; ++r) v[r] = x[r];
          const float top = rows_max(v, lane);
          if (lane % (32 / RP) == 0)
            reinterpret_cast<float *>(&sh->red[t & 1][lane / (32 / RP)])[warp] = top;
        }
        ok = named_barrier_and(kBarSoftmax, kSoftmaxThreads, ok && okw);
        if (!ok) break;
        // the lazy running maximum (identical in every thread)
        float alpha[RP];
        bool rescale = false;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float4 w = sh->red[t & 1][r];
          const float tm = fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w));
          const bool up = tm > m[r] + kRescaleThreshold;
          const bool moved = up && m[r] != -INFINITY;
          alpha[r] = moved ? ex2_approx(m[r] - tm) : 1.f;
          l[r] *= alpha[r];
          rescale |= moved;
          m[r] = up ? tm : m[r];
        }
        if (rescale) {
          // O holds PV products of earlier tiles of this part: wait for the
          // last one (PV_{t-1}), then scale its columns
          const int u = t - 1;
          const bool okr = mbar_wait_warp(&sh->pv_done[u & 1], (u >> 1) & 1, abort_flag, p.wait_ns);
          if (okr) {
            tc_fence_after();
            const uint32_t ta = tmem + lane_base + 2 * kN + (oi & 1) * C::kOCols + o_col;
#pragma unroll
            for (int two = 0; two < (C::kTwo ? 2 : 1); ++two) {
              uint32_t o[RP];
              tmem_ld_cols(ta + two * C::kLo, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < RP; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c]);
              tmem_st_cols(ta + two * C::kLo, o);
            }
            tmem_wait_st();
          }
          ok = okr;
        }
        // P buffer t % 2 held P_{t-2}: its product must be done reading it
        if (t >= 2 && ok)
          ok = mbar_wait_warp(&sh->pv_done[t & 1], ((t - 2) >> 1) & 1, abort_flag, p.wait_ns);
        // row r of P_t: keys of this tile, bf16, 128B-swizzled rows; the second
        // 64 keys kPHalf further (the second half of the d = 64 product's rows)
        const uint32_t pb = smem_addr(pbuf + (t & 1) * C::kPBytes) + (k >> 6) * C::kPHalf;
        const uint32_t kc = static_cast<uint32_t>(k & 63);
        auto p_at = [&](int r) { return pb + r * 128 + (((kc >> 3) ^ (r & 7)) << 4) + (kc & 7) * 2; };
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float pr = ex2_approx(x[r] - (m[r] == -INFINITY ? 0.f : m[r]));
          l[r] += pr;
          const uint16_t hi = bf16_bits(pr);
          st_shared_u16(p_at(r), hi);
          if (C::kTwo)
            st_shared_u16(p_at(r + C::kLo),
                          bf16_bits(pr - __uint_as_float(static_cast<uint32_t>(hi) << 16)));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sh->p_full[t & 1]);
        ++t;
        if (++slot == C::kSlots) {
          slot = 0;
          ++round;
        }
      }
      // All four gave up at a tile's barrier.  (A warp alone may have in its waits behind the
      // last one: it meets the others at the barrier below, where all learn of it.)
      if (j < d.tiles) break;
      // ---- l = sum over the key slots; O = O^T / l, or both as they are -----
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float v = warp_sum(l[r]);
        if (lane == 0) reinterpret_cast<float *>(&sh->lsum[r])[warp] = v;
      }
      const int u = t - 1;
      const bool oke =
          ok && mbar_wait_warp(&sh->pv_done[u & 1], (u >> 1) & 1, abort_flag, p.wait_ns);
      // d = 64: the second key half's output goes through the P buffer of the last
      // tile, which its product has read
      float *xo = reinterpret_cast<float *>(pbuf + (u & 1) * C::kPBytes);
      uint32_t o[RP];
      if (oke) {
        tc_fence_after();
        const uint32_t ta = tmem + lane_base + 2 * kN + (oi & 1) * C::kOCols + o_col;
        tmem_ld_cols(ta, o);
        if (C::kTwo) {
          uint32_t lo[RP];
          tmem_ld_cols(ta + C::kLo, lo);
          tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < RP; ++r) {
            // (an infinite value: what the rounding left, of either sign, times infinity)
            const float a = __uint_as_float(o[r]), b = __uint_as_float(lo[r]);
            o[r] = __float_as_uint(fabsf(a) == INFINITY ? a : a + b);
          }
        } else {
          tmem_wait_ld();
        }
        if (D == 64 && warp >= 2) {
#pragma unroll
          for (int r = 0; r < RP; ++r) xo[r * 64 + vdim] = __uint_as_float(o[r]);
        }
      }
      tc_fence_before();
      mbar_arrive(&sh->o_free[oi & 1]);
      ++oi;
      ok = named_barrier_and(kBarSoftmax, kSoftmaxThreads, oke);
      if (!ok) break;
      if (stores) {
        float *sums = d.slot >= 0 ? paged_slot_ptr(p, D, blockIdx.x, d.slot) : nullptr;
        // Row r's sum, and what it is divided by, in lane r (and those r + RP, ...): one
        // quotient to a warp.  (Row after row in every thread, the output of 8 rows took 3000
        // cycles.)
        const int own = lane & (RP - 1);
        const float4 ls = sh->lsum[own];
        float lt = (ls.x + ls.y) + (ls.z + ls.w), mt = m[0];
#pragma unroll
        for (int r = 1; r < RP; ++r) mt = own == r ? m[r] : mt;
        if (sums == nullptr && mt == kLowestScore) lt = NAN;
        const float inv = 1.f / lt;
        const unsigned none = __ballot_sync(0xffffffffu, lt == 0.f);  // no allowed key: +0.0
        float acc[RP];
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          acc[r] = __uint_as_float(o[r]);
          if (D == 64) acc[r] += xo[r * 64 + vdim];
        }
        int h = 0, i = 0;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          const float f = __shfl_sync(0xffffffffu, inv, r);
          if (r < R && h < d.heads && i < d.tokens) {
            if (sums != nullptr) {
              sums[r * D + vdim] = acc[r];
              if (k == r) {  // (of warp 0)
                sums[p.rows * D + 2 * r] = mt;
                sums[p.rows * D + 2 * r + 1] = lt;
              }
            } else {
              out[row_at(h, i) * D + vdim] = bf16_bits((none >> r) & 1 ? 0.f : acc[r] * f);
            }
          }
          if (++i == p.tb) {
            i = 0;
            ++h;
          }
        }
      }
      // lsum and that P buffer are rewritten only after the next part's first
      // tile barrier, which every thread reaches after the reads above
    }
  }

  // ---- teardown --------------------------------------------------------------
  if (*abort_flag && warp == 4 && lane == 0) {
    for (int idx = issued - C::kSlots; idx < issued; ++idx)
      if (idx >= 0) (void)wait_teardown(&sh->kv_full[idx % C::kSlots], (idx / C::kSlots) & 1);
    for (int qi = q_issued - 2; qi < q_issued; ++qi)
      if (qi >= 0) (void)wait_teardown(&sh->q_full[qi & 1], (qi >> 1) & 1);
  }
  if (*abort_flag && (warp == 5 || warp == 6) && lane == 0 && last_commit != nullptr)
    (void)wait_teardown(last_commit, last_parity);
  if (*abort_flag && threadIdx.x == 0) atomicExch(p.status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int RP, bool kTree>
cudaError_t launch_as(const FewMaps &maps, const PagedProblem &p, int &grid, int num_sms,
                        cudaStream_t stream) {
  using C = Cfg<D, RP>;
  constexpr size_t kSmem = smem_bytes<D, RP>();
  // 1 KB per CTA is the system's
  static_assert(RP * 64 * sizeof(float) <= C::kPBytes, "output of a key half in a P buffer");
  static_assert(C::kCtas * (kSmem + 1024) <= 233472, "shared memory budget");
  static_assert(C::kSlots <= kMaxSlots, "ring size");
  grid = std::min(grid, C::kCtas * num_sms);
  const cudaError_t e = set_smem_once(
      reinterpret_cast<const void *>(paged_few_tc_kernel<D, RP, kTree>), static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_few_tc_kernel<D, RP, kTree>, maps, p);
}

template <int D, int RP>
cudaError_t launch_impl(const FewMaps &maps, const PagedProblem &p, int &grid, int num_sms,
                        cudaStream_t stream) {
  return p.tree != nullptr ? launch_as<D, RP, true>(maps, p, grid, num_sms, stream)
                           : launch_as<D, RP, false>(maps, p, grid, num_sms, stream);
}

template <int D>
cudaError_t launch_rows(const FewMaps &maps, const PagedProblem &p, int &grid, int num_sms,
                        cudaStream_t stream) {
  const int R = p.hpu * p.tb;
  if (R <= 1) return launch_impl<D, 1>(maps, p, grid, num_sms, stream);
  if (R <= 2) return launch_impl<D, 2>(maps, p, grid, num_sms, stream);
  if (R <= 4) return launch_impl<D, 4>(maps, p, grid, num_sms, stream);
  if (R <= 8) return launch_impl<D, 8>(maps, p, grid, num_sms, stream);
  return launch_impl<D, 16>(maps, p, grid, num_sms, stream);
}

}  // namespace

cudaError_t launch_paged_few(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                             const PagedProblem &p, int d, int &grid, int num_sms,
                             cudaStream_t stream) {
  if (p.hpu * p.tb > kN) return cudaErrorInvalidValue;
  const FewMaps maps{q, k, v};
  return d == 128 ? launch_rows<128>(maps, p, grid, num_sms, stream)
                  : launch_rows<64>(maps, p, grid, num_sms, stream);
}

}  // namespace mha

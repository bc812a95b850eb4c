// Attention of many query rows against a paged key/value cache on the tcgen05
// tensor cores (bf16, d in {64, 128}): chunks of prompts, drafted tokens of many
// heads, batches that mix chunks and single tokens.
//
// A part of work (paged.cuh) is up to 256 query rows of one key/value head -- its
// group's query heads times `tb` tokens -- against some 128-key tiles.  Packing the
// group's heads into the rows reads each key once for all of them.  Two softmax
// warpgroups own a 128-row TMEM tile each:
//
//   S_w = Q_w K_j^T      tcgen05.mma, both operands 128B-swizzled in smem
//   softmax              thread = row; the running maximum moves only when it grows
//                        by more than 2^8 (numerator and denominator share it)
//   P_w (bf16) -> TMEM   over S_w's first columns.  Weights are rounded to nearest
//                        (2^-8 relative): a second bf16 for what the rounding
//                        leaves would add half again to the products that bound
//                        the kernel
//   O_w += P_w V_j       A = P_w from TMEM, B = V_j from smem
//
// While one warpgroup turns its S into P the tensor core runs the other's products.
// With tokens for one 128-row tile at most, both warpgroups take the same rows, the
// even and the odd tiles, and join their sums at the end of the part: a lone
// warpgroup would leave the tensor core and the loads waiting for its softmax.
//
// Bound: the tensor cores for long chunks (4 d flop per row and key), HBM for short
// chunks behind long caches.  Persistent CTAs, one per SM, take equal stretches of
// all units' tiles (causal limits counted), cutting a unit's keys where a stretch
// ends; paged_merge_rows_kernel joins the cut ones.  Tiles come page by page as in
// paged_few_tc.cu; value rows behind the part's last key, or of pages that are not
// there, are zeroed in shared memory by a warp of their own before the product
// reads them.
//
// Measured, with the merge: a prompt of 8192 tokens, 16 heads, d 128: 223 us, 1.23
// PFLOP/s of allowed products (0.65 of a library product's rate); 8 chunks of up to 512
// tokens behind 1000-4096 keys, 32 heads over 8: 78 us, 0.73 PFLOP/s; 4 x 4096 tokens, 16
// heads, d 64: 215 us, 0.64 PFLOP/s.  A pair of tiles takes about 1.75 us at d 128 and
// 1.55 at d 64, whose products are half as long, so the chain of a row sets the pace: one
// thread's two passes over 128 columns (0.85 us), then its two products, which have to
// wait because P_w lies in S_w's columns.  d = 64 has columns for P of its own, but scores
// formed before the products then cost more in waits than they gain (215 -> 227 us).  The
// way to the first tile is 8 us, a part's beginning and end 3, the merge 6.  Up to 32 rows
// (drafts of grouped heads) lie in one warp of a warpgroup, and the others wait for its
// exponentials: 16 x 8 tokens over 4000 keys, 32 heads over 8, d 128: 63 us, 0.62 of HBM.
// Trees of drafted tokens (kTree: the row's mask words are looked at in a sequence's last
// tiles only): 16 of 9-25 tokens behind 1000-4096 keys, 32 heads over 8, d 128: 49 us, 3.5
// TB/s (6 us to the first tile, then 1.67 a tile, 2 to 3 to a part's output, merge 5); 64 of
// 64 tokens behind 4096-8192: 327 us, 1.25 PFLOP/s, 0.76 of HBM (1.76 us a pair of tiles,
// which HBM brings in 1.47); 256 of 8 tokens behind 128-1024, 3 to 9 tiles to a unit: 175
// us, 0.54 of HBM, 4 us between one part's last tile and the next part's first.  Two
// warpgroups to a tile, 64 columns each, were slower (327 -> 383 us): 104 registers do not
// hold a thread's scores, and every more wait for TMEM is 250 cycles.
//
// Warp roles (384 threads): warps 0-3 and 4-7 softmax, warp 8 producer (walks the
// parts and hands their descriptions to the others), warp 9 TMEM owner and product
// issuer, warp 10 zeroes value rows, warp 11 completes the third warpgroup, whose
// registers go to the softmax.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace mha {
namespace {

constexpr int kBN = kPagedTile;
constexpr int kThreads = 384;
constexpr int kWgThreads = 128;
// Register split: 384 threads launched at 168 each; the control warpgroup drops
// to 72 and the softmax warpgroups rise to 216: 2 x 128 x 216 + 128 x 72 = 384 x 168.
constexpr uint32_t kRegsSoftmax = 216;
constexpr uint32_t kRegsControl = 72;
static_assert(2 * 128 * kRegsSoftmax + 128 * kRegsControl <= kThreads * 168, "register split");
constexpr uint32_t kTmemCols = 512;        // S_w at 128 w, O_w at 256 + 128 w
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr float kFarScore = 16777216.f;    // 2^24
constexpr int kMaxSlots = 8;
constexpr int kDescs = 4;     // part descriptions in flight
constexpr int kPresent = 16;  // tiles whose pages' presence is kept (more than are in flight)

template <int D>
struct Cfg {
  static constexpr int kSlabs = D / 64;
  static constexpr int kBlkBytes = 128 * 128;            // one [128 rows x 64] swizzle block
  static constexpr int kTileBytes = kSlabs * kBlkBytes;  // a [128 x D] operand tile
  static constexpr int kSlots = D == 128 ? 5 : 8;        // K/V ring (K0 V0 K1 V1 ...)
};

// A part as the other roles need it.
struct Desc {
  int go;        // 0: no more parts
  int tiles;     // of the part (0: rows of zeros)
  int tiles0;    // of warpgroup 0, when the warpgroups have rows of their own
  int both;      // the warpgroups share the rows and take every other tile
  int key0;      // first key of the first tile
  int kv_end;    // keys from here on are not attended to
  int lim0;      // keys below this are allowed for the first token
  int lim_step;  // ... plus this per token
  int row0;      // first row of q and out
  int tokens, heads, h0;
  int slot;      // of its sums; -1: the part is a whole unit
};

struct __align__(16) Shared {
  float joined[2][kWgThreads];  // warpgroup 1's (max, sum) of rows that both have
  long long scratch[40];
  Desc desc[kDescs];
  uint32_t present[kPresent];  // pages of a tile that were loaded
  int zero_slot, zero_rows;    // for the zeroing warp: V slot (-1: done), rows below are whole
  uint32_t zero_present;       // ... pages that were loaded
  int steps;                   // loads that the producer has come to
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  uint64_t q_full, q_empty;
  uint64_t kv_full[kMaxSlots], kv_empty[kMaxSlots];
  uint64_t v_landed;           // copies of a V tile that the zeroing warp finishes
  uint64_t zero_full, zero_empty;
  uint64_t s_full[2];   // S_w of the next tile (and every product before it)
  uint64_t p_full[2];   // P_w written
  uint64_t pv_done[2];  // last P_w V of a part
  uint64_t o_free[2];   // O_w of a part has been read
  uint64_t join;        // `joined` is written
  uint64_t drain;       // teardown: every tcgen05 operation of the CTA has finished
  uint32_t tmem_base;
  int abort_flag;
};

template <int D>
constexpr size_t smem_bytes() {
  using C = Cfg<D>;
  return 1024 + static_cast<size_t>(2 + C::kSlots) * C::kTileBytes + sizeof(Shared);
}

struct ManyMaps {
  CUtensorMap q;     // (d, T, H, 1), box (64, tb / 2, hpu, 1)
  CUtensorMap k, v;  // (d, page_size, H_kv, num_pages), box (64, min(page_size, 128), 1, 1)
};

// Row maximum of one 32-column chunk (raw fp32 bits); a tree of 3-input maxima.
__device__ __forceinline__ float chunk_max32(const uint32_t (&v)[32]) {
  float t[11];
#pragma unroll
  for (int k = 0; k < 10; ++k)
    t[k] = fmax3(__uint_as_float(v[3 * k]), __uint_as_float(v[3 * k + 1]),
                 __uint_as_float(v[3 * k + 2]));
  t[10] = fmaxf(__uint_as_float(v[30]), __uint_as_float(v[31]));
  return fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]),
               fmax3(fmax3(t[6], t[7], t[8]), t[9], t[10]));
}

// p_c = exp2(s_c * sl - m) for one 32-column chunk, packed into 16 bf16x2
// columns; returns the chunk's sum of p (fp32)
__device__ __forceinline__ float chunk_exp_pack32(const uint32_t (&v)[32], float sl, float m,
                                                  uint32_t (&pk)[16]) {
  const uint64_t sc = f2_pack(sl, sl);
  const uint64_t nm = f2_pack(-m, -m);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float a, b;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc, nm), a, b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(a, b));
    pk[e >> 1] = pack_bf16x2(a, b);
  }
  acc[0] = f2_add(acc[0], acc[1]);
  acc[2] = f2_add(acc[2], acc[3]);
  acc[0] = f2_add(acc[0], acc[2]);
  float lo, hi;
  f2_unpack(acc[0], lo, hi);
  return lo + hi;
}

// Multiplies the 32 bf16 P values of one chunk (16 TMEM columns) by f, after
// the stores in flight have landed.
__device__ __noinline__ void rescale_p16(uint32_t taddr, float f) {
  uint32_t r[16];
  tmem_wait_st();
  tmem_ld16(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int t = 0; t < 16; ++t)
    r[t] = pack_bf16x2(__uint_as_float(r[t] << 16) * f, __uint_as_float(r[t] & 0xffff0000u) * f);
  tmem_st16(taddr, r);
}

__device__ __forceinline__ void st_global_v8(void *to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Stores the warp's 32 rows of O (TMEM o0 times a0, plus TMEM o1 times a1): as fp32
// to rows `mine` of a slot of sums, or as bf16 to rows `mine` of out (-1: no row of
// ours).  A store's time is that of the 128-byte lines it touches: a slot holds its
// rows' columns four by four ([d / 4][rows][4]; a warp's store is 512 bytes in a
// stretch), and out is written 32 bytes a lane where it is aligned to that.
// kNoTmem stands for zeros; `none`: this lane's row is zeros whatever TMEM holds.
constexpr uint32_t kNoTmem = 0xffffffffu;
template <int D>
__device__ __forceinline__ void store_rows(uint32_t o0, uint32_t o1, float a0, float a1, bool none,
                                           int mine, float *slot, int rows, uint16_t *out) {
  const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    uint32_t o[32];
    if (o0 != kNoTmem) {
      tmem_ld32(o0 + c0, o);
      tmem_wait_ld();
    }
#pragma unroll
    for (int e = 0; e < 32; ++e)
      o[e] = o0 == kNoTmem || none ? 0u : __float_as_uint(__uint_as_float(o[e]) * a0);
    if (o1 != kNoTmem) {
#pragma unroll
      for (int hf = 0; hf < 32; hf += 16) {
        uint32_t t[16];
        tmem_ld16(o1 + c0 + hf, t);
        tmem_wait_ld();
        if (!none) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[hf + e] =
                __float_as_uint(fmaf(__uint_as_float(t[e]), a1, __uint_as_float(o[hf + e])));
        }
      }
    }
    if (mine >= 0 && slot != nullptr) {
      float *to = slot + (static_cast<size_t>(c0 / 4) * rows + mine) * 4;
#pragma unroll
      for (int e = 0; e < 32; e += 4, to += static_cast<size_t>(rows) * 4)
        st_global_v4(to, make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
    } else if (mine >= 0) {
      uint16_t *to = out + static_cast<size_t>(mine) * D + c0;
#pragma unroll
      for (int e = 0; e < 32; e += 16) {
        uint32_t v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[k] = pack_bf16x2(__uint_as_float(o[e + 2 * k]), __uint_as_float(o[e + 2 * k + 1]));
        if (wide) {
          st_global_v8(to + e, v);
        } else {
          st_global_v4(to + e, make_uint4(v[0], v[1], v[2], v[3]));
          st_global_v4(to + e + 8, make_uint4(v[4], v[5], v[6], v[7]));
        }
      }
    }
  }
}

template <int D, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
    paged_many_tc_kernel(const __grid_constant__ ManyMaps maps,
                         const __grid_constant__ PagedProblem p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *q_smem = smem;                         // 2 tiles
  uint8_t *kv_smem = q_smem + 2 * C::kTileBytes;  // kSlots tiles
  Shared *sh = reinterpret_cast<Shared *>(kv_smem + C::kSlots * C::kTileBytes);
  volatile int *abort_flag = &sh->abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tbw = p.tb >> 1;  // tokens of a warpgroup's tile

  // ---- setup -------------------------------------------------------------
  if (threadIdx.x == 0) {
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sh->kv_full[s], 1);
      mbar_init(&sh->kv_empty[s], 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&sh->desc_full[i], 1);
      mbar_init(&sh->desc_empty[i], 9);  // eight softmax warps, the issuer
    }
    mbar_init(&sh->v_landed, 1);
    mbar_init(&sh->zero_full, 1);
    mbar_init(&sh->zero_empty, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sh->s_full[w], 1);
      mbar_init(&sh->p_full[w], kWgThreads);
      mbar_init(&sh->pv_done[w], 1);
      mbar_init(&sh->o_free[w], kWgThreads);
    }
    mbar_init(&sh->join, kWgThreads);
    mbar_init(&sh->drain, 1);
    sh->steps = 0;
    sh->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 9) {
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

  int issued = 0, zeroed = 0, q_issued = 0;  // producer: ring loads, handed-over V tiles, Q loads
  bool mma_issued = false;                   // issuer: a product was issued

  if (warp >= 8) {
    regs_dec<kRegsControl>();
    if (warp == 8) {
      // ---- producer: walks the parts; per part Q, then K_j V_j K_j+1 ... ----
      const PagedBatch &pb = p.batch;
      const int box = min(pb.page_size, kBN);  // rows of a copy
      const int pieces_shift = 7 - min(pb.page_shift, 7);
      const int pieces = 1 << pieces_shift;    // copies per 64 columns of a tile
      const bool loads = lane < C::kSlabs * pieces;
      const int piece = lane & (pieces - 1);
      const int slab = loads ? lane >> pieces_shift : 0;
      const int dst0 = slab * C::kBlkBytes + piece * box * 128;
      const uint32_t whole = (1u << pieces) - 1;
      // Lane 0 walks, one part ahead of the loads, so that the other roles find the
      // next part's description when they get there.  The walk and the two parts live
      // in shared memory (where the span was found), out of this warpgroup's few
      // registers.
      PagedWalk &walk = *reinterpret_cast<PagedWalk *>(&sh->scratch[0]);
      PagedPart *const two = reinterpret_cast<PagedPart *>(&sh->scratch[14]);
      static_assert(sizeof(PagedWalk) <= 14 * 8 && 14 * 8 + 2 * sizeof(PagedPart) <= 32 * 8,
                    "where they live");
      if (lane == 0) walk.begin(p, span);
      int n = 0, flags = 0, mrow = 0, mtokens = 0, mhead = 0, mheads = 0;
      bool ok = true, more = false;
      // the description of the part in two[n & 1], or of the end
      auto describe = [&]() {
        const PagedPart &part = two[n & 1];
        const bool got = more;
        ok = mbar_wait_warp(&sh->desc_empty[n % kDescs], ((n / kDescs) & 1) ^ 1, abort_flag,
                            p.wait_ns);
        if (!ok) return;
        if (lane == 0) {
          const bool split = got && paged_split(part);
          Desc d;
          d.go = got;
          d.tiles = part.t1 - part.t0;
          const int end0 = paged_kv_end(part.seq, min(part.i0 + tbw, part.i1), p.causal);
          d.tiles0 = max(min((end0 + kBN - 1) / kBN, part.t1) - part.t0, 0);
          d.both = part.i1 - part.i0 <= tbw;
          d.key0 = part.t0 * kBN;
          d.kv_end = part.kv_end;
          // of a tree: where its tokens begin
          d.lim0 =
              kTree ? part.seq.base : (p.causal ? part.seq.base + part.i0 + 1 : part.seq.len);
          d.lim_step = p.causal;
          d.row0 = part.seq.q0 + part.i0;
          d.tokens = part.i1 - part.i0;
          d.heads = part.heads;
          d.h0 = part.h0;
          d.slot = split ? paged_slot(part) : -1;
          sh->desc[n % kDescs] = d;
          mbar_arrive(&sh->desc_full[n % kDescs]);
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
        __syncwarp();
        ++n;
      };
      // the part whose tiles are being loaded: tiles [j, t1) are left
      int j = 0, t1 = 0, kv_end = 0, head = 0, id = -1;
      const int32_t *table = nullptr;
      // page of this lane's copies of tile j; -1 when it holds no key or is not there
      auto page_of = [&](int tile) -> int {
        const int key = tile * kBN + piece * box;
        if (!loads || tile >= t1 || key >= kv_end) return -1;
        const int at = table[key >> pb.page_shift];
        return static_cast<unsigned>(at) < static_cast<unsigned>(pb.num_pages) ? at : -1;
      };
      while (ok) {
        // the next part, into two[n & 1] (the one at hand is two[(n - 1) & 1])
        more = __any_sync(0xffffffffu, lane == 0 && walk.next(p, two[n & 1]));
        __syncwarp();
        // the rest of the part at hand, then the first tile of the next one (this loop
        // has one copy of the code that issues a tile: it competes with the softmax for
        // the instruction cache)
#pragma unroll 1
        for (int phase = 0; phase < 2 && ok; ++phase) {
          int stop = t1;
          if (phase == 1) {
            if (!more) break;
            const PagedPart &part = two[n & 1];
            j = stop = t1 = 0;
            if (part.nt == 0) break;
            j = part.t0;
            t1 = part.t1;
            stop = j + 1;
            kv_end = part.kv_end;
            head = part.kv;
            table = pb.block_table + static_cast<size_t>(part.b) * pb.max_pages;
            id = page_of(j);
            ok = mbar_wait_warp(&sh->q_empty, (q_issued & 1) ^ 1, abort_flag, p.wait_ns);
            if (!ok) break;
            if (lane == 0) {
              const int halves = part.i1 - part.i0 <= tbw ? 1 : 2;
              mbar_arrive_expect_tx(&sh->q_full,
                                    static_cast<uint32_t>(halves * C::kSlabs * tbw * p.hpu * 128));
              for (int w = 0; w < halves; ++w)
                for (int blk = 0; blk < C::kSlabs; ++blk)
                  tma_load_4d(q_smem + w * C::kTileBytes + blk * C::kBlkBytes, &maps.q,
                              &sh->q_full, blk * 64, part.seq.q0 + part.i0 + w * tbw, part.h0, 0);
            }
            ++q_issued;
          }
          for (; j < stop && ok; ++j) {
            const int id_next = page_of(j + 1);
            const uint32_t there = __ballot_sync(0xffffffffu, id >= 0) & whole;
            const uint32_t bytes = static_cast<uint32_t>(__popc(there) * box * 128 * C::kSlabs);
            const int rows = min(kv_end - j * kBN, kBN);
            const int row_in_page = (j * kBN + piece * box) & (pb.page_size - 1);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {  // K, then V
              const int slot = issued % C::kSlots, round = issued / C::kSlots;
              ok = mbar_wait_warp(&sh->kv_empty[slot], (round & 1) ^ 1, abort_flag, p.wait_ns);
              if (!ok) break;
              uint64_t *bar = &sh->kv_full[slot];
              const bool partial = kv == 1 && (there != whole || rows < kBN);
              if (partial) {
                // the zeroing warp announces this tile once its rows are finished
                bar = &sh->v_landed;
                ok = mbar_wait_warp(&sh->zero_empty, (zeroed & 1) ^ 1, abort_flag, p.wait_ns);
                if (!ok) break;
                ++zeroed;
              }
              if (lane == 0) {
                if (kv == 0) {
                  *const_cast<volatile int *>(&sh->steps) = issued;
                  sh->present[(issued >> 1) % kPresent] = there;
                } else if (partial) {
                  sh->zero_slot = slot;
                  sh->zero_rows = rows;
                  sh->zero_present = there;
                  mbar_arrive(&sh->zero_full);
                }
                mbar_arrive_expect_tx(bar, bytes);
              }
              __syncwarp();
              if (id >= 0)
                tma_load_4d(kv_smem + slot * C::kTileBytes + dst0, kv == 0 ? &maps.k : &maps.v,
                            bar, slab * 64, row_in_page, head, id);
              ++issued;
            }
            id = id_next;
          }
        }
        // (after its first loads are on their way)
        if (ok) describe();
        if (!more) break;
      }
      if (ok && mbar_wait_warp(&sh->zero_empty, (zeroed & 1) ^ 1, abort_flag, p.wait_ns) &&
          lane == 0) {
        sh->zero_slot = -1;
        mbar_arrive(&sh->zero_full);
      }
      if (lane == 0) {
        int32_t *meta = p.meta + static_cast<size_t>(blockIdx.x) * kPagedMeta;
        meta[kMetaFlags] = flags;
        meta[kMetaRow] = mrow;
        meta[kMetaTokens] = mtokens;
        meta[kMetaHead] = mhead;
        meta[kMetaHeads] = mheads;
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---- issuer: lane 0 alone (tcgen05.mma and commit are single-thread
      // instructions); the other lanes wait at the end --------------------------
      // step i of a part, per warpgroup w: O_w += P_w(i-1) V(i-1), then S_w(i) = Q_w K(i)
      if (lane == 0) {
        const uint32_t idesc_s = idesc_bf16_f32(128, kBN, 0);
        const uint32_t idesc_o = idesc_bf16_f32(128, D, 1);
        const uint32_t hi = smem_desc_hi(1024);  // of every operand
        const uint32_t q_lo = smem_desc_lo(smem_addr(q_smem), 16);
        const uint32_t k_lo = smem_desc_lo(smem_addr(kv_smem), 16);
        const uint32_t v_lo = smem_desc_lo(smem_addr(kv_smem), C::kBlkBytes);
        constexpr uint32_t kTileLo = C::kTileBytes >> 4;
        int n = 0, nq = 0;           // descriptions and non-empty parts so far
        int tw[2] = {0, 0};          // tiles of each warpgroup so far
        int pw[2] = {0, 0};          // parts with tiles of each warpgroup so far
        int base = 0;                // ring index of the part's first K
        bool ok = true;
        while (ok) {
          ok = mbar_wait_spin(&sh->desc_full[n % kDescs], (n / kDescs) & 1, abort_flag, p.wait_ns);
          if (!ok) break;
          const int go = sh->desc[n % kDescs].go, tiles = sh->desc[n % kDescs].tiles;
          const int tiles0 = sh->desc[n % kDescs].tiles0, both = sh->desc[n % kDescs].both;
          mbar_arrive(&sh->desc_empty[n % kDescs]);
          ++n;
          if (!go) break;
          if (tiles == 0) continue;
          // test hook: a wait on a barrier that nothing signals before the teardown; in every
          // other CTA before its first product, in the others with a part's behind it
          if ((p.stall & kStallPagedManyMma) != 0 && nq == static_cast<int>(blockIdx.x & 1) &&
              !(ok = mbar_wait_spin(&sh->drain, 0, abort_flag, p.wait_ns)))
            break;
          ok = mbar_wait_spin(&sh->q_full, nq & 1, abort_flag, p.wait_ns);
          const int cnt[2] = {both ? (tiles + 1) >> 1 : tiles0, both ? tiles >> 1 : tiles};
          const int steps = max(cnt[0], cnt[1]);
          // ring positions of K(i) and V(i-1) of each warpgroup, stepped without divisions
          int ks[2], kr[2], vs[2], vr[2];
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int at = base + (both ? 2 * w : 0);
            ks[w] = at % C::kSlots;
            kr[w] = at / C::kSlots;
            vs[w] = (at + 1) % C::kSlots;
            vr[w] = (at + 1) / C::kSlots;
          }
          const int stride = both ? 4 : 2;
          // the first key step of O's product overwrites O when `first`
          auto pv = [&](int slot, int w, bool first) {
            uint32_t lo = v_lo + slot * kTileLo;
            asm volatile("" : "+r"(lo));
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk) {
              tc_mma_ts(tmem + 256 + w * 128, tmem + w * 128 + kk * 8, desc_join(lo, hi), idesc_o,
                        !first || kk > 0);
              lo += (16 * 128) >> 4;
            }
          };
          auto score = [&](int slot, int w, int q_tile) {
            uint32_t lo = k_lo + slot * kTileLo, ql = q_lo + q_tile * kTileLo;
            asm volatile("" : "+r"(lo), "+r"(ql));
#pragma unroll 1
            for (int blk = 0; blk < C::kSlabs; ++blk) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_ss(tmem + w * 128, desc_join(ql + kk * 2, hi), desc_join(lo + kk * 2, hi),
                          idesc_s, blk > 0 || kk > 0);
              ql += C::kBlkBytes >> 4;
              lo += C::kBlkBytes >> 4;
            }
            tc_commit(&sh->s_full[w]);
          };
          auto step = [&](int &slot, int &round) {
            slot += stride;
            if (slot >= C::kSlots) {
              slot -= C::kSlots;
              ++round;
            }
          };
          mma_issued = true;
          for (int i = 0; ok && i <= steps; ++i) {
            if (!both && i >= 2 && i < cnt[0]) {
              // an inner step of rows of their own: nothing but the products and their
              // waits (this thread sets the kernel's pace)
              if (!(ok = mbar_wait_spin(&sh->kv_full[vs[0]], vr[0] & 1, abort_flag, p.wait_ns)))
                break;
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                if (!(ok = mbar_wait_spin(&sh->p_full[w], (tw[w] + i - 1) & 1, abort_flag,
                                          p.wait_ns)))
                  break;
                tc_fence_after();
                pv(vs[0], w, false);
                if (w == 0 && !(ok = mbar_wait_spin(&sh->kv_full[ks[0]], kr[0] & 1, abort_flag,
                                                    p.wait_ns)))
                  break;
                score(ks[0], w, w);
              }
              if (!ok) break;
              if (i == steps - 1) tc_commit(&sh->q_empty);
              step(vs[0], vr[0]);
              step(ks[0], kr[0]);
              vs[1] = vs[0];
              vr[1] = vr[0];
              ks[1] = ks[0];
              kr[1] = kr[0];
              continue;
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const bool do_pv = i >= 1 && i - 1 < cnt[w];
              const bool do_s = i < cnt[w];
              // a tile that the other warpgroup waited for is there
              const bool waits = both || w == 0;
              if (do_pv) {
                if ((waits || i - 1 >= cnt[0]) &&
                    !(ok = mbar_wait_spin(&sh->kv_full[vs[w]], vr[w] & 1, abort_flag, p.wait_ns)))
                  break;
                if (!(ok = mbar_wait_spin(&sh->p_full[w], (tw[w] + i - 1) & 1, abort_flag,
                                          p.wait_ns)))
                  break;
                // the part's first product overwrites O: it has been read
                if (i == 1 &&
                    !(ok = mbar_wait_spin(&sh->o_free[w], (pw[w] & 1) ^ 1, abort_flag, p.wait_ns)))
                  break;
                tc_fence_after();
                pv(vs[w], w, i == 1);
                if (i == cnt[w]) tc_commit(&sh->pv_done[w]);
                step(vs[w], vr[w]);
              }
              if (do_s && (waits || i >= cnt[0]) &&
                  !(ok = mbar_wait_spin(&sh->kv_full[ks[w]], kr[w] & 1, abort_flag, p.wait_ns)))
                break;
              if (do_s) {
                score(ks[w], w, both ? 0 : w);
                step(ks[w], kr[w]);
              }
            }
            if (ok && i == steps - 1) tc_commit(&sh->q_empty);  // every S of the part is issued
          }
          base += 2 * tiles;
          ++nq;
          for (int w = 0; w < 2; ++w) {
            tw[w] += cnt[w];
            pw[w] += cnt[w] > 0;
          }
        }
      }
      __syncwarp();
    } else if (warp == 10) {
      // ---- finishes V tiles whose last rows, or some pages, were not loaded ----
      const int box_shift = min(p.batch.page_shift, 7);
      for (int n = 0;; ++n) {
        // (tiles that need finishing may be few: a chunk of whole tiles has none)
        if (!mbar_wait_idle(&sh->zero_full, n & 1, abort_flag, p.wait_ns, &sh->steps)) break;
        const int slot = sh->zero_slot, rows = sh->zero_rows;
        const uint32_t there = sh->zero_present;
        if (slot < 0) break;
        if (!mbar_wait_warp(&sh->v_landed, n & 1, abort_flag, p.wait_ns)) break;
        const uint32_t v = smem_addr(kv_smem + slot * C::kTileBytes);
        // eight lanes per row
        for (int r = lane >> 3; r < kBN; r += 4)
          if (r >= rows || !((there >> (r >> box_shift)) & 1))
            for (int s = 0; s < C::kSlabs; ++s)
              st_shared_v4(v + s * C::kBlkBytes + r * 128 + (lane & 7) * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->kv_full[slot]);
          mbar_arrive(&sh->zero_empty);
        }
        __syncwarp();
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ---- softmax warpgroups --------------------------------------------------
    const int w = warp >> 2;          // warpgroup
    const int r = threadIdx.x & 127;  // row within the tile (TMEM lane)
    const int head = r / tbw, tok = r - head * tbw;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lane_base + w * 128;
    const uint32_t o_tmem = tmem + lane_base + 256 + w * 128;
    const int box_shift = min(p.batch.page_shift, 7);
    const uint32_t whole = (1u << (kBN >> box_shift)) - 1;
    const bool pos = p.scale_log2 > 0.f;  // the max over scaled scores is the scaled max
    uint16_t *out = static_cast<uint16_t *>(p.out);
    int ts = 0;        // tiles of this warpgroup so far
    int parts[2] = {0, 0};  // parts with tiles of each warpgroup so far
    int joins = 0;
    int tile0 = 0;     // tiles of the CTA before the part
    bool ok = true;
    for (int n = 0;; ++n) {
      ok = mbar_wait_warp(&sh->desc_full[n % kDescs], (n / kDescs) & 1, abort_flag, p.wait_ns);
      if (!ok) break;
      const Desc d = sh->desc[n % kDescs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->desc_empty[n % kDescs]);
      if (!d.go) break;
      const int i = (d.both ? 0 : w * tbw) + tok;  // token of the unit
      const bool row = head < d.heads && i < d.tokens && head < p.hpu;
      const size_t out_row = static_cast<size_t>(d.row0 + i) * p.H + d.h0 + head;
      const int cnt = d.both ? (d.tiles + 1 - w) >> 1 : (w == 0 ? d.tiles0 : d.tiles);
      const bool join = d.both && d.tiles > 1;  // warpgroup 1 has sums of the same rows
      const bool live_warp = __any_sync(0xffffffffu, row);
      // keys below jmax are allowed for this row
      const int jmax = min(d.lim0 + i * d.lim_step, d.kv_end);
      const bool releaser = (d.both || w == 1) && r == 0;

      float m_use = -INFINITY;  // max used for the exponentials (log2 units)
      float l_run = 0.f;
      for (int it = 0; it < cnt; ++it) {
        const int jj = d.both ? 2 * it + w : it;  // tile of the part
        // Of a tree: the row's words that this tile needs, loaded before the wait; only a
        // sequence's last tiles need any.
        uint32_t words[5] = {0u, 0u, 0u, 0u, 0u};
        const int from = d.key0 + jj * kBN - d.lim0;
        if (kTree && row && from > -kBN) {
          const uint32_t *tree = p.tree + static_cast<size_t>(d.row0 + i) * p.tree_words;
#pragma unroll
          for (int x = 0; x < 5; ++x) words[x] = tree_word(tree, p.tree_words, (from >> 5) + x);
        }
        // S_w is ready, and so is every product issued before it (same commit)
        if (!(ok = mbar_wait_warp(&sh->s_full[w], ts & 1, abort_flag, p.wait_ns))) break;
        tc_fence_after();
        if (releaser) {
          const int k_at = 2 * (tile0 + jj);
          mbar_arrive(&sh->kv_empty[k_at % C::kSlots]);
          if (it > 0) mbar_arrive(&sh->kv_empty[(k_at + (d.both ? -3 : -1)) % C::kSlots]);
        }
        ++ts;
        if (!live_warp) {  // no row of this warp is anyone's: its P and O stay whatever they are
          tc_fence_before();
          mbar_arrive(&sh->p_full[w]);
          continue;
        }
        const int key = d.key0 + jj * kBN;
        const int lim = min(max(jmax - key, 0), kBN);
        const uint32_t there = sh->present[(tile0 + jj) % kPresent];
        // pages that are not there, among those that hold keys of the part
        const uint32_t holes =
            whole & ~there & ((2u << ((min(d.kv_end - key, kBN) - 1) >> box_shift)) - 1);
        const bool need_mask = holes != 0 || __any_sync(0xffffffffu, lim < kBN);
        // Two passes over the scores: their maximum, then the weights against the running
        // one, which moves only when it grows by more than 2^8.  Reading the scores twice
        // costs less than taking 32 columns' maximum and weights in turn (234 -> 225 us on
        // a prompt of 8192 tokens, 16 heads, d 128).  P of 32 columns goes to 16, whose
        // scores have been read; it is handed over whole (by halves, the products waited
        // for one warpgroup while the other's were ready: 260 us).  Loops, not straight
        // code: the roles' loops together have to stay in the instruction cache (305 -> 243
        // us on 4 x 4096 tokens, 16 heads, d 64, with the products' loops from 183 to 94
        // KB).
        float alpha = 1.f, tsum = 0.f;
        bool plain = pos && !need_mask;
        uint32_t v[2][32];
        float cm = -INFINITY;
        if (plain) {
          // (the first 64 columns last: the second pass begins with them)
#pragma unroll 1
          for (int ch = 2; ch >= 0; ch -= 2) {
            tmem_ld32(s_tmem + ch * 32, v[0]);
            tmem_ld32(s_tmem + ch * 32 + 32, v[1]);
            tmem_wait_ld();
            cm = fmax3(cm, chunk_max32(v[0]), chunk_max32(v[1]));
          }
          cm = fmaxf(cm * p.scale_log2, kLowestScore);
          // The weights' exponents come from one fused product and difference, which the
          // rounding of the maximum shifts by up to 2^-24 of it: the same for a row's weights
          // and their sum, but past 2^31 enough to leave the range of fp32.  Such scores take
          // the other way.
          const bool climb = cm > m_use + kRescaleThreshold, far = fabsf(cm) > kFarScore;
          if (__any_sync(0xffffffffu, climb || far)) {
            plain = !__any_sync(0xffffffffu, far);
            if (plain && climb) {
              alpha = ex2_approx(m_use - cm);
              m_use = cm;
            }
          }
        }
        if (plain) {
#pragma unroll 1
          for (int ch = 0; ch < 4; ch += 2) {
            if (ch > 0) {
              tmem_ld32(s_tmem + ch * 32, v[0]);
              tmem_ld32(s_tmem + ch * 32 + 32, v[1]);
              tmem_wait_ld();
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t pk[16];
              tsum += chunk_exp_pack32(v[k], p.scale_log2, m_use, pk);
              tmem_st16(s_tmem + (ch + k) * 16, pk);
            }
          }
        } else {
          // masks, holes, far scores, a scale that is not positive: scores scaled (the max of
          // scale * s is not scale * max s) and masked first; in one pass, for these tiles
          // are few.  A chunk whose max exceeds the running one rescales the P of the
          // chunks already stored.
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t(&v0)[32] = v[0];
            tmem_ld32(s_tmem + ch * 32, v0);
            // columns of the chunk's two halves that count: below the limit, and not of
            // a page that is not there (pages have at least 16 rows)
            const int upto = (kTree ? min(d.kv_end - key, kBN) : lim) - ch * 32;
            const int upto0 = (holes >> ((ch * 32) >> box_shift)) & 1 ? 0 : upto;
            const int upto1 = (holes >> ((ch * 32 + 16) >> box_shift)) & 1 ? 0 : upto;
            uint32_t see = 0xffffffffu;
            if (kTree) {
              see = tree_window(words[0], words[1], from + ch * 32);
#pragma unroll
              for (int x = 0; x < 4; ++x) words[x] = words[x + 1];
              see &= (upto0 >= 16 ? 0xffffu : (1u << max(upto0, 0)) - 1u) |
                     ((upto1 >= 32 ? 0xffffu : (1u << max(upto1 - 16, 0)) - 1u) << 16);
            }
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              v0[e] = __float_as_uint((kTree ? (see >> e) & 1u : e < (e < 16 ? upto0 : upto1))
                                          ? __uint_as_float(v0[e]) * p.scale_log2
                                          : -INFINITY);
            cm = chunk_max32(v0);
            // a key is seen
            if (kTree ? see != 0 : upto0 > 0 || upto1 > 16) cm = fmaxf(cm, kLowestScore);
            const bool climb = cm > m_use + kRescaleThreshold;
            if (__any_sync(0xffffffffu, climb)) {
              const float f = climb ? ex2_approx(m_use - cm) : 1.f;
              if (climb) m_use = cm;
              alpha *= f;
              tsum *= f;
#pragma unroll 1
              for (int c = 0; c < ch; ++c) rescale_p16(s_tmem + c * 16, f);
            }
            uint32_t pk[16];
            // no key so far: weights of 0, not of -inf less -inf
            tsum += chunk_exp_pack32(v0, 1.f, m_use == -INFINITY ? 0.f : m_use, pk);
            tmem_st16(s_tmem + ch * 16, pk);
          }
        }
        l_run = l_run * alpha + tsum;
        // the running max moved: rescale this row of O (rare, warp-wide)
        if (it > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tmem_ld32(o_tmem + ch * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(o_tmem + ch * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh->p_full[w]);
      }
      if (!ok) break;
      if (cnt > 0) {
        ok = mbar_wait_warp(&sh->pv_done[w], parts[w] & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        if (releaser) {
          const int last = tile0 + (d.both ? 2 * (cnt - 1) + w : cnt - 1);
          mbar_arrive(&sh->kv_empty[(2 * last + 1) % C::kSlots]);
        }
      }
      tile0 += d.tiles;

      // ---- output: O / l, or O and its statistics as they are --------------------
      float f0 = 1.f, f1 = 0.f;
      if (d.both && w == 1) {
        // warpgroup 0 writes these rows.  It has read what was joined before: this
        // part's first product into O_1 waited for that (o_free)
        if (join) {
          sh->joined[0][r] = m_use;
          sh->joined[1][r] = l_run;
          mbar_arrive(&sh->join);
          ++parts[1];
        }
        continue;
      }
      if (join) {
        ok = mbar_wait_warp(&sh->join, joins & 1, abort_flag, p.wait_ns) &&
             mbar_wait_warp(&sh->pv_done[1], parts[1] & 1, abort_flag, p.wait_ns);
        if (!ok) break;
        ++joins;
        const float m1 = sh->joined[0][r], l1 = sh->joined[1][r];
        const float mt = fmaxf(m_use, m1), use = mt == -INFINITY ? 0.f : mt;
        f0 = ex2_approx(m_use - use);
        f1 = ex2_approx(m1 - use);
        l_run = l_run * f0 + l1 * f1;
        m_use = mt;
      }
      tc_fence_after();
      parts[0] += d.both ? cnt > 0 : d.tiles0 > 0;
      parts[1] += d.both ? join : d.tiles > 0;
      const int unit_row = head * p.tb + i;
      float *slot = d.slot >= 0 ? paged_slot_ptr(p, D, blockIdx.x, d.slot) : nullptr;
      if (slot != nullptr && row) {
        float *ml = slot + static_cast<size_t>(p.rows) * D + 2 * unit_row;
        ml[0] = m_use;
        ml[1] = l_run;
      }
      if (slot == nullptr && m_use == kLowestScore) l_run = NAN;
      const bool none = l_run == 0.f;  // nothing attended to: +0.0
      const float inv = slot != nullptr ? 1.f : (none ? 0.f : 1.f / l_run);
      const int mine = row ? (slot != nullptr ? unit_row : static_cast<int>(out_row)) : -1;
      if (live_warp)
        store_rows<D>(cnt > 0 ? o_tmem : kNoTmem, join ? o_tmem + 128 : kNoTmem,
                      none ? 0.f : f0 * inv, none ? 0.f : f1 * inv, none, mine, slot, p.rows, out);
      tc_fence_before();
      if (cnt > 0) mbar_arrive(&sh->o_free[w]);
      if (join) mbar_arrive(&sh->o_free[1]);  // warpgroup 1's, with its statistics
    }
  }

  // ---- teardown --------------------------------------------------------------
  if (*abort_flag && warp == 8 && lane == 0) {
    for (int idx = issued - C::kSlots; idx < issued; ++idx)
      if (idx >= 0) (void)wait_teardown(&sh->kv_full[idx % C::kSlots], (idx / C::kSlots) & 1);
    if (zeroed > 0) (void)wait_teardown(&sh->v_landed, (zeroed - 1) & 1);
    if (q_issued > 0) (void)wait_teardown(&sh->q_full, (q_issued - 1) & 1);
  }
  if (*abort_flag && warp == 9 && lane == 0 && mma_issued) {
    // tcgen05 ops of one thread complete in order: one more commit covers
    // every product issued before it
    tc_commit(&sh->drain);
    (void)wait_teardown(&sh->drain, 0);
  }
  if (*abort_flag && threadIdx.x == 0) atomicExch(p.status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool kTree>
cudaError_t launch_as(const ManyMaps &maps, const PagedProblem &p, int grid,
                        cudaStream_t stream) {
  constexpr size_t kSmem = smem_bytes<D>();
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(Cfg<D>::kSlots <= kMaxSlots && Cfg<D>::kSlots > 4, "ring size");
  // setmaxnreg.inc only succeeds if the launch reserved the registers it hands
  // out; refuse to launch a build whose register count would not cover them
  // (checked once per process: the register count is a property of the build)
  static std::atomic<int> regs_ok{0};  // 0 unknown, 1 enough, 2 too few
  if (regs_ok.load(std::memory_order_acquire) == 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, paged_many_tc_kernel<D, kTree>);
    if (e != cudaSuccess) return e;
    regs_ok.store(static_cast<long long>(fa.numRegs) * kThreads >=
                          2LL * 128 * kRegsSoftmax + 128LL * kRegsControl
                      ? 1
                      : 2,
                  std::memory_order_release);
  }
  if (regs_ok.load(std::memory_order_acquire) != 1) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      set_smem_once(reinterpret_cast<const void *>(paged_many_tc_kernel<D, kTree>),
                    static_cast<int>(kSmem));
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
  return cudaLaunchKernelEx(&cfg, paged_many_tc_kernel<D, kTree>, maps, p);
}

template <int D>
cudaError_t launch_impl(const ManyMaps &maps, const PagedProblem &p, int grid,
                        cudaStream_t stream) {
  return p.tree != nullptr ? launch_as<D, true>(maps, p, grid, stream)
                           : launch_as<D, false>(maps, p, grid, stream);
}

}  // namespace

cudaError_t launch_paged_many(const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                              const PagedProblem &p, int d, int grid, cudaStream_t stream) {
  if (p.hpu * (p.tb / 2) > 128) return cudaErrorInvalidValue;
  const ManyMaps maps{q, k, v};
  return d == 128 ? launch_impl<128>(maps, p, grid, stream) : launch_impl<64>(maps, p, grid, stream);
}

}  // namespace mha

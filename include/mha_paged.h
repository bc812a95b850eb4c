/*
 * mha_paged.h -- C ABI of the operators around the attention of a decoder that
 * generates from a paged key/value cache, and of their training counterpart:
 *
 *   mha_qk_norm_rope_fwd   per-head RMS norm of queries and keys and the
 *                          position rotation, in one pass
 *   mha_qk_norm_rope_bwd   its gradients
 *   mha_paged_append       the same for new tokens of ragged sequences, the
 *                          keys and values going into the pages of a cache
 *   mha_paged_fwd          attention of the new tokens over the paged cache
 *   mha_paged_append_at    mha_paged_append with given positions: drafted trees
 *   mha_paged_tree_fwd     attention of trees of drafted tokens
 *   mha_paged_compact      the tokens that stay, moved to the front or elsewhere
 *   mha_paged_reserve      the page tables of the next step: sequences that grow,
 *                          shrink, fork, end and begin
 *   mha_paged_copy         pages copied to pages, in all layers
 *
 * A generation step is mha_linear_fwd (the projections), mha_paged_append,
 * mha_paged_fwd, mha_linear_fwd; one that verifies drafted trees takes
 * mha_paged_append_at and mha_paged_tree_fwd instead, and mha_paged_compact when
 * it knows which drafted tokens it accepts.  mha_paged_reserve and mha_paged_copy
 * come before either, and once more behind mha_paged_compact, to give back the pages
 * that only rejected tokens took.  The pages that mha.h cites describe a decoder
 * that attends to every earlier position (alexdo.xyz, "How predictions are
 * generated"); paging, rotation and head norms are how present decoders carry
 * that out, and have no counterpart on the pages.
 *
 * Conventions are those of mha.h: device pointers owned by the caller,
 * contiguous row-major tensors, 16-byte aligned unless said otherwise; every
 * call enqueues its work on `stream` and returns; nothing is allocated and
 * nothing is synchronised; errors found in the arguments return before anything
 * is enqueued.  Lengths, offsets, positions and page numbers are read on the
 * device; whatever they hold, no access leaves the buffers the arguments
 * describe.  The library keeps no state between calls, and two calls may run at
 * once (other streams, threads or devices) as long as they share no workspace
 * and no buffer that one of them writes.
 */
#ifndef MHA_GB300_PAGED_H
#define MHA_GB300_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "mha.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which dimensions of a head form the pairs that are rotated (r = rotary_dim). */
enum {
  MHA_ROPE_HALVES = 0,      /* (i, i + r/2), i < r/2 */
  MHA_ROPE_INTERLEAVED = 1  /* (2i, 2i + 1),  i < r/2 */
};

/*
 * mha_qk_norm_rope_fwd -- between the projections and the attention:
 *
 *     n = x / sqrt(mean_c x_c^2 + eps) * weight        (each head's row x of d)
 *     y_a = n_a cos(p f_i) - n_b sin(p f_i)
 *     y_b = n_a sin(p f_i) + n_b cos(p f_i)            (pair i = (a, b))
 *
 * for every row of q and k, p its position and f_i = inv_freq[i]; dimensions
 * from rotary_dim on keep n.  Arithmetic in fp32, one rounding at the end; the
 * angle p f_i is reduced in 64-bit fixed point, so far positions lose nothing.
 *
 * q [B, H, L, d], k [B, H_kv, L, d] (MHA_LAYOUT_BHSD) or [B, L, heads, d]
 *               (MHA_LAYOUT_BSHD); dtype F32 or BF16; d is 64 or 128
 * q_out, k_out  like q and k; each may be its input itself (in place), and
 *               overlaps no other argument
 * q_weight, k_weight  [d] in dtype, or NULL: that tensor's rows are not normed
 * positions     int32 [B, L], 4-byte aligned, or NULL for 0 .. L - 1; any value
 * inv_freq      fp32 [rotary_dim / 2], 4-byte aligned, finite, |f| < 2^20
 *               (ignored when rotary_dim is 0)
 * B, H, H_kv, L >= 0; a tensor without elements is ignored (its pointers may be
 *               NULL), e.g. H_kv = 0 for queries alone; H_kv need not divide H.
 *               B * L and H + 2 H_kv are at most 2^31 - 2^20 - 1
 * rotary_dim    0 .. d, a multiple of 16
 * style         MHA_ROPE_HALVES or MHA_ROPE_INTERLEAVED
 * eps           finite, >= 0
 */
int mha_qk_norm_rope_fwd(const void *q, const void *k, void *q_out, void *k_out,
                         const void *q_weight, const void *k_weight, const int32_t *positions,
                         const float *inv_freq, int B, int H, int H_kv, int L, int d,
                         int rotary_dim, int layout, int style, float eps, int dtype,
                         void *stream);

/* Bytes of device workspace mha_qk_norm_rope_bwd needs (partial sums of the
   weights' gradients); 0 for a d it does not support. */
size_t mha_qk_norm_rope_bwd_workspace_size(int d);

/*
 * mha_qk_norm_rope_bwd -- gradients of a loss through mha_qk_norm_rope_fwd.
 * With g the incoming gradient rotated back and r = 1 / sqrt(mean x^2 + eps):
 *
 *     dweight = sum over all rows of g x r
 *     dx = r (weight g - x r mean_c(weight g x r))
 *
 * (dx = g where that tensor's weight is NULL).
 *
 * q, k, weights, positions, inv_freq and the numbers: those of the forward call
 *               (q and k are not read where the weight is NULL: may be NULL)
 * dq_out, dk_out  dL/dq_out and dL/dk_out, like q and k
 * dq, dk        results like q and k, overwritten; each may be its incoming
 *               gradient itself (in place), and overlaps no other argument
 * dq_weight, dk_weight  results, fp32 [d], overwritten; NULL exactly where the
 *               weight is NULL.  Sums run in a fixed order: the same inputs on
 *               the same device give the same bits.  Zero where a tensor has no
 *               rows.
 * workspace     device memory of at least mha_qk_norm_rope_bwd_workspace_size(d)
 *               bytes, 256-byte aligned, overlapping nothing (not read, and may
 *               be NULL, when both weights are NULL); scratch afterwards
 */
int mha_qk_norm_rope_bwd(const void *q, const void *k, const void *dq_out, const void *dk_out,
                         void *dq, void *dk, float *dq_weight, float *dk_weight,
                         const void *q_weight, const void *k_weight, const int32_t *positions,
                         const float *inv_freq, int B, int H, int H_kv, int L, int d,
                         int rotary_dim, int layout, int style, float eps, int dtype,
                         void *workspace, size_t workspace_bytes, void *stream);

/*
 * Ragged batches and the paged cache (mha_paged_append, mha_paged_fwd)
 *
 * A batch holds B sequences whose new tokens lie behind one another in the rows
 * of q, k, v and out:
 *
 * q_starts    int32 [B + 1]: sequence b's new tokens are rows q_starts[b] ..
 *             q_starts[b + 1] - 1.  Not decreasing, within [0, T]; values
 *             outside are clamped.  Rows before q_starts[0] and from
 *             q_starts[B] on belong to no sequence and are left as they were.
 * kv_lengths  int32 [B]: the sequence's length in the cache, its new tokens
 *             among them: new token i (of n) sits at position
 *             p = kv_lengths[b] - n + i.  Negative: 0.
 * block_table int32 [B, max_pages]: position p of sequence b lives in page
 *             block_table[b][p / page_size] at p % page_size.  Entries that hold
 *             no position of the sequence are not read.  An entry outside
 *             [0, num_pages) names no page: its positions are neither written
 *             nor attended to, nor are positions from max_pages * page_size on.
 * k_cache, v_cache  [num_pages, H_kv, page_size, d] (MHA_LAYOUT_BHSD) or
 *             [num_pages, page_size, H_kv, d] (MHA_LAYOUT_BSHD).  Cells that
 *             hold no position of a sequence may contain anything.  Sequences
 *             may share pages that they only read.
 *
 * T * H and B * H are at most 2^31 - 1 (mha_paged_fwd); T and H + 2 H_kv at most
 * 2^31 - 2^20 - 1 (mha_paged_append).  More is MHA_ERR_UNSUPPORTED.
 *
 * These three arrays are 4-byte aligned.  page_size is a power of two >= 16;
 * d is 64 or 128; H_kv divides H; dtype F32 or BF16 for every tensor.
 */

/*
 * mha_paged_append -- the norm and rotation of mha_qk_norm_rope_fwd for the new
 * tokens of a ragged batch, each at its position p; keys and values go into the
 * cache.
 *
 * q, q_out  [T, H, d]; q_out may be q itself; both NULL with H = 0: keys and
 *           values alone
 * k, v      [T, H_kv, d]
 * A token whose position is negative or lies in no page has no row in the cache
 * and is skipped there; its q_out row is written all the same.  Two tokens of a
 * call must not share a cell (the cell would hold one of them, or parts of
 * both).  Other arguments as above; rotary_dim = 0 and NULL weights only copy.
 */
int mha_paged_append(const void *q, const void *k, const void *v, void *q_out, void *k_cache,
                     void *v_cache, const void *q_weight, const void *k_weight,
                     const float *inv_freq, const int32_t *q_starts, const int32_t *kv_lengths,
                     const int32_t *block_table, int B, int T, int H, int H_kv, int d,
                     int num_pages, int page_size, int max_pages, int rotary_dim, int layout,
                     int style, float eps, int dtype, void *stream);

/*
 * mha_paged_append_at -- mha_paged_append whose rotation angles are those of given
 * positions: a token of a drafted tree is rotated at the position it would have
 * (the cached length plus its depth), and written to the cell of its place among
 * the new tokens.
 *
 * positions  int32 [T]: row t is rotated by positions[t] f_i; any value, not read
 *            for rows of no sequence.  Everything else as above: cells are those
 *            of p = kv_lengths[b] - n + i.
 */
int mha_paged_append_at(const void *q, const void *k, const void *v, void *q_out, void *k_cache,
                        void *v_cache, const void *q_weight, const void *k_weight,
                        const float *inv_freq, const int32_t *positions, const int32_t *q_starts,
                        const int32_t *kv_lengths, const int32_t *block_table, int B, int T, int H,
                        int H_kv, int d, int num_pages, int page_size, int max_pages,
                        int rotary_dim, int layout, int style, float eps, int dtype, void *stream);

/* Bytes of device workspace mha_paged_fwd needs for these arguments, whatever
   the lengths (sums of sequences whose keys are split over the GPU); 0 for
   arguments it would reject or an empty problem. */
size_t mha_paged_workspace_size(int B, int T, int H, int H_kv, int d, int max_q, int dtype);

/*
 * mha_paged_fwd -- attention of the new tokens over the paged cache:
 *
 *     out[t,h,:] = sum_j softmax_j( scale * q[t,h,:] . k_j ) v_j
 *
 * over the positions j of token t's sequence, key/value head h / (H / H_kv).
 *
 * q, out     [T, H, d]; out overlaps no other argument
 * mask_kind  MHA_MASK_CAUSAL_TAIL: token i sees positions j <= kv_lengths[b] - n + i;
 *            MHA_MASK_NONE: it sees all kv_lengths[b] positions
 * max_q      the most new tokens of a sequence that the caller expects, >= 1 (1
 *            for a step of single tokens).  It chooses the kernel, and the result
 *            is right whatever it is; a good value is the largest
 *            q_starts[b + 1] - q_starts[b].  (BF16: up to (H / H_kv) max_q = 8 the
 *            softmax weights are kept to 2^-17, past that to 2^-8.)
 * scale      finite
 * max_pages * page_size  at most 2^31 - 1024
 * workspace  device memory of at least mha_paged_workspace_size(...) bytes,
 *            256-byte aligned, overlapping nothing; scratch afterwards
 *
 * A position that a token does not see adds nothing to it whatever its key
 * holds; its value must be finite where a later token of the same call sees it
 * (a weight of 0 times infinity is NaN). Tokens with nothing to attend to are
 * written as +0.0, whatever their query holds. What a token does see counts as
 * the formula says: a NaN in its query or in such a key, a score past the range
 * of fp32, or scores all of which are -infinity make its row NaN; a score of
 * -infinity beside others weighs nothing. Sums and softmax statistics are fp32;
 * with BF16 the softmax weights are rounded to bfloat16 for the product with
 * the values.
 */
int mha_paged_fwd(const void *q, const void *k_cache, const void *v_cache, void *out,
                  const int32_t *q_starts, const int32_t *kv_lengths, const int32_t *block_table,
                  int B, int T, int H, int H_kv, int d, int max_q, int num_pages, int page_size,
                  int max_pages, int layout, int mask_kind, float scale, int dtype,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * mha_paged_tree_fwd -- mha_paged_fwd for drafted tokens that form trees: token i of
 * a sequence's n new ones sees every position before the first new token, and of
 * the new ones those that the mask names (its ancestors, and itself).
 *
 * tree_mask  int32 [T, tree_words], 4-byte aligned: bit m % 32 of word m / 32 of
 *            row t says whether token t sees new token m of its sequence (position
 *            kv_lengths[b] - n + m).  Bits from n on mean nothing; new tokens from
 *            32 tree_words on are seen by none.  Any bits are allowed, none too:
 *            what a row sees need not be a path, and a row that sees nothing (and
 *            has nothing cached before the new tokens) is written as +0.0.
 * tree_words >= 1
 * The workspace is that of mha_paged_fwd.  The kernel is the one that mha_paged_path
 * tells, but where there is little work for what the block table has room for, 4 or 8 rows are
 * taken at a time, with BF16 on the few-query kernel (no call tells; a wider table may take
 * longer over the same lengths); everything else as there (a new token's value must be finite
 * where any other token of its sequence is in the call).  With BF16 the softmax weights are
 * kept to 2^-17 where 8 rows or fewer are taken at a time, else to 2^-8, as there.
 */
int mha_paged_tree_fwd(const void *q, const void *k_cache, const void *v_cache, void *out,
                       const int32_t *tree_mask, const int32_t *q_starts,
                       const int32_t *kv_lengths, const int32_t *block_table, int B, int T, int H,
                       int H_kv, int d, int max_q, int num_pages, int page_size, int max_pages,
                       int tree_words, int layout, float scale, int dtype, void *workspace,
                       size_t workspace_bytes, void *stream);

/* Which kernel mha_paged_fwd would launch: 0 = none (empty problem), 1 = fp32
   CUDA-core kernel, 2 = few-query tensor-core kernel (at most 16 expected query
   rows, (H / H_kv) * max_q, per key/value head), 3 = many-query tensor-core
   kernel; negative = -(mha_status) for arguments it would reject.  Host only. */
int mha_paged_path(int B, int T, int H, int H_kv, int d, int max_q, int page_size, int dtype);

/*
 * The page pool
 *
 * The operators below work on the block tables themselves and, for the caches of
 * `layers` layers that lie behind one another in memory, on [layers, num_pages, ...]
 * with every layer's pages laid out as above.  A sequence has the same pages in every
 * layer and in both caches.  All int32 arrays are 4-byte aligned; the caches 16-byte.
 */

/* Bytes of device workspace mha_paged_reserve needs; 0 for arguments it rejects. */
size_t mha_paged_reserve_workspace_size(int B, int num_pages);

/*
 * mha_paged_reserve -- the block tables of the next step.  Row i of the new tables
 * continues row parents[i] of the old ones: it keeps the first
 * keep = min(kv_lengths[parents[i]], new_lengths[i]) positions and gets pages for
 * new_lengths[i].  So a sequence grows (parents[i] = i, a larger length), gives
 * back what rejected tokens took (a smaller one), ends (0), begins (parents[i] = -1)
 * or forks (a parent that several rows name, as beams do).
 *
 * kv_lengths say how far the old tables reach: pages that hold positions below them are
 * given up, what a table names behind them is not.  They are the lengths_out of the call
 * that made the tables, also when the sequences have become shorter since: with the lengths
 * that mha_paged_compact leaves, the pages behind those would be held for ever.  So a step
 * whose drafted tokens are decided ends with a call that has the reach as kv_lengths, the
 * lengths that are left as new_lengths and no parents.  Where no row forks, the call that
 * begins the next step can do it as well: the reach as kv_lengths, the next lengths as
 * new_lengths (the rows keep pages of rejected tokens as far as they need them, and write over
 * them; rows that fork would share those pages).
 *
 * refs counts each page's references: one for every row that holds a position in
 * it, and whatever the caller adds to hold on to a page (a cached prefix).  With
 * whole pages shared, and a part-filled last page a row's own, because the row will
 * write to it:
 *
 *   refs_out[p] = refs[p] - references of the old rows + whole pages of the new rows
 *   Where keep is no multiple of page_size, row i keeps its last page p if
 *   refs_out[p] is then 0 or less and i is the lowest row whose last page p is, and
 *   refs_out[p] grows by one.  Other such rows need a copy: a new page in p's place,
 *   and moves[i] = (p, new page) for mha_paged_copy (otherwise (-1, -1)).
 *   Pages with refs_out <= 0 are free.  The rows in their order get the lowest-numbered
 *   free ones: a row's copy first, then the pages its new positions need, ascending.
 *   They get refs_out = 1.
 *
 * When the free pages run out, the remaining places hold -1 and lengths_out says
 * how far the row's pages go: new_lengths[i] where it got them all (at most
 * max_pages * page_size), else the positions in the pages it has (without its
 * part-filled page when that one's copy is missing).  The inputs are left as they
 * were (but for refs where refs_out is refs), so the caller may choose other lengths
 * and call again.
 *
 * block_table, kv_lengths  int32 [B_old, max_pages], [B_old]: the old tables and how far
 *               they reach; entries outside [0, num_pages) name no page, and are -1 where
 *               they are kept
 * new_lengths, parents  int32 [B], [B]; a parent outside [0, B_old) is none; NULL:
 *               row i's is i.  Lengths below 0 count as 0, those past
 *               max_pages * page_size as that
 * refs, refs_out  int32 [num_pages]; refs_out may be refs itself
 * table_out, lengths_out, moves  int32 [B, max_pages], [B], [B, 2], overwritten;
 *               entries that hold no position are -1
 * counts        int32 [2], or NULL: pages given out, pages free after it
 * B_old, B, num_pages at most 2^31 - 2^20 - 1, B_old * max_pages and
 *               B * (max_pages + 1) at most 2^29 - 1, max_pages * page_size at most
 *               2^31 - 1024
 * workspace     device memory of at least mha_paged_reserve_workspace_size(B,
 *               num_pages) bytes, 256-byte aligned, overlapping nothing
 */
int mha_paged_reserve(const int32_t *block_table, const int32_t *kv_lengths,
                      const int32_t *new_lengths, const int32_t *parents, const int32_t *refs,
                      int32_t *table_out, int32_t *lengths_out, int32_t *refs_out, int32_t *moves,
                      int32_t *counts, int B_old, int B, int num_pages, int page_size,
                      int max_pages, void *workspace, size_t workspace_bytes, void *stream);

/*
 * mha_paged_copy -- k_cache[l, moves[i][1]] = k_cache[l, moves[i][0]], and v_cache,
 * for every layer l and pair i (those of mha_paged_reserve).
 *
 * k_cache, v_cache  [layers, num_pages, page_size * H_kv * d], either layout
 * moves    int32 [n, 2]; a pair with a number outside [0, num_pages) is skipped.  A
 *          page that is written is no other pair's page (it would hold one of what
 *          the pairs say, or parts of both)
 */
int mha_paged_copy(void *k_cache, void *v_cache, const int32_t *moves, int n, int layers, int H_kv,
                   int d, int num_pages, int page_size, int dtype, void *stream);

/*
 * mha_paged_compact -- the tokens that stay of each sequence: position
 * starts[b] + keep[b][i] moves to position starts[b] + i, in every layer, and the
 * sequence ends behind the last:
 *
 *     lengths_out[b] = starts[b] + the number of kept tokens
 *
 * An accepted path of a drafted tree (starts: the cached length before the tree,
 * keep: its tokens' numbers), or what is left of a long sequence.  The sequence holds its
 * pages as far as kv_lengths until mha_paged_reserve, told those, gives them back.
 *
 * keep        int32 [B, max_keep], keep_counts [B] (clamped to [0, max_keep]): a list
 *             ascends, from 0 on, and stays below kv_lengths[b] - starts[b].  It ends
 *             before the first entry that does not (an entry that is no larger than the
 *             one before it, a position that the sequence does not have)
 * starts      int32 [B], or NULL: 0.  Clamped to [0, kv_lengths[b]]
 * kv_lengths  int32 [B]: the lengths before; negative: 0
 * block_table int32 [B, max_pages]: the pages that are written
 * src_table   like it: the pages that are read; NULL, or block_table itself: in place.
 *             Otherwise no cell that is written is read as well, by any sequence (a token
 *             whose cell is the same in both tables is neither read nor written)
 * A position in no page is neither read nor written.  In place, what a cell held is read
 * before it is written; cells that are written belong to one sequence (and one place of
 * its table) only.  lengths_out overlaps nothing.
 * 2 B H_kv layers is at most 2^31 - 1, max_keep 2^30
 */
int mha_paged_compact(void *k_cache, void *v_cache, int32_t *lengths_out, const int32_t *keep,
                      const int32_t *keep_counts, const int32_t *starts,
                      const int32_t *kv_lengths, const int32_t *src_table,
                      const int32_t *block_table, int B, int layers, int H_kv, int d,
                      int num_pages, int page_size, int max_pages, int max_keep, int layout,
                      int dtype, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MHA_GB300_PAGED_H */

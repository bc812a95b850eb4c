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
 *
 * A generation step is mha_linear_fwd (the projections), mha_paged_append,
 * mha_paged_fwd, mha_linear_fwd.  The pages that mha.h cites describe a decoder
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

/* Which kernel mha_paged_fwd would launch: 0 = none (empty problem), 1 = fp32
   CUDA-core kernel, 2 = few-query tensor-core kernel (at most 16 expected query
   rows, (H / H_kv) * max_q, per key/value head), 3 = many-query tensor-core
   kernel; negative = -(mha_status) for arguments it would reject.  Host only. */
int mha_paged_path(int B, int T, int H, int H_kv, int d, int max_q, int page_size, int dtype);

#ifdef __cplusplus
}
#endif

#endif /* MHA_GB300_PAGED_H */

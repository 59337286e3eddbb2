/*
 * rfpx_verify.h -- C ABI of librfpx, verification of drafted tokens: a step
 * brings every sequence a tree of columns, and leaves it the drafts that the
 * model itself would have written.
 *
 *   rfpx_tree_masks         parents turned into ancestor bits and positions
 *   rfpx_attn_tree_forward  attention of a tree's columns over the FP4 cache
 *   rfpx_sample             a token for every column from its logits
 *   rfpx_tree_accept        the drafts that the drawn tokens confirm
 *   rfpx_kv_commit          their keys and values moved together in the cache
 *
 * The conventions of rfpx.h hold, cache and batch are those of rfpx_attn.h
 * (rfpx_kv_append writes a tree's columns as it does any step's).
 *
 * ------------------------------------------------------------- the tree
 * Of a sequence's n columns (rows starts[b] .. starts[b+1]-1) column 0 is the
 * token that was settled last and the others are drafts.  parents[row] is the
 * column, of the same sequence and before this one, that a column follows;
 * -1, or a number that is no such column, makes it one that follows the
 * context alone.  A sequence may have no columns, and at most
 * RFPX_TREE_COLS_MAX of them; rows of columns behind that, rows at or behind
 * starts[n_seqs] and at or behind n_rows are neither read nor written, except
 * that rfpx_attn_tree_forward computes any number of columns.
 *
 * rfpx_tree_masks and rfpx_tree_accept have no cache and take lens as it
 * stands, past pages_per_seq * page_tokens and below 0 too.  The other calls
 * count it as that, or as 0: of a sequence that has outgrown its pages lens has
 * to be set to what they hold before the step, or the two would go on from
 * slots that are not there.
 */
#ifndef RFPX_VERIFY_H
#define RFPX_VERIFY_H

#include "rfpx_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RFPX_TREE_COLS_MAX 1024
#define RFPX_VOCAB_MAX (1 << 20)

/* For every row, from parents_dev [n_rows]:
 *   masks[row][w]   bit j of word w: column 32 w + j is this column or one of
 *                   its ancestors (uint32 [n_rows][mask_words]; columns past
 *                   32 * mask_words have no bit)
 *   positions[row]  base[b] plus the number of its ancestors (int32; NULL:
 *                   not written)
 * base_dev int32 [n_seqs]: the position of column 0; NULL: lens[b] - n, its
 * slot.  1 <= mask_words <= RFPX_TREE_COLS_MAX / 32. */
rfpx_status rfpx_tree_masks(const rfpx_kv_batch *b, int n_rows, const int32_t *parents_dev,
                            const int32_t *base_dev, int mask_words, uint32_t *masks_dev,
                            int32_t *positions_dev, void *stream);

/* Workspace of rfpx_attn_tree_forward; 0 if unsupported.  As
 * rfpx_attn_workspace_bytes. */
size_t rfpx_attn_tree_workspace_bytes(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int n_heads,
                                      int n_rows);

/* rfpx_attn_forward with other slots seen: column i of n sees slots 0 ..
 * lens[b] - n - 1, and of the step's slots lens[b] - n + j those whose bit j
 * is set in masks_dev [n_rows][mask_words] (its own among them: the bits alone
 * decide; bits of columns that do not exist, and columns that have no bit, are
 * not seen).  A column whose own slot is negative sees nothing.  Everything
 * else is as rfpx_attn_forward has it.  (rfpx_attn_weights takes a step's columns
 * as a chain: it has no form for trees.) */
rfpx_status rfpx_attn_tree_forward(const rfpx_kv_cache *c, const rfpx_kv_batch *b,
                                   const void *q_dev, long long q_stride, int xtype, int n_heads,
                                   int n_rows, float scale, const uint32_t *masks_dev,
                                   int mask_words, void *out_dev, long long out_stride,
                                   float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream);

/* Workspace of rfpx_sample; 0 if unsupported.  256-byte aligned, no
 * initialization needed, scratch between calls. */
size_t rfpx_sample_workspace_bytes(int n_rows, int vocab, int xtype);

/* A token of every row of logits [n_rows][vocab] (fp32 or bf16 per xtype, rows
 * `stride` elements apart, any alignment of a whole element), drawn by the
 * row's number u in [0, 1).  The tokens of a row are ordered by logit, the
 * largest first, ties by the lower index, and weigh
 *   w = exp((logit - largest) / temperature).
 * Of this order stay
 *   the first top_k (0 or less: all),
 *   of those the fewest first ones whose weights sum to top_p of theirs (not
 *   below 1: all; 0 or less: the first),
 *   of those the ones of w >= min_p (above 1 counts as 1),
 * always the first one among them, and the token drawn is the first whose
 * weight, summed up with those before it, exceeds u times the sum of all that
 * stay.  tokens_dev int32 [n_rows] gets its index, probs_dev (fp32, or NULL)
 * its weight over that sum.  A temperature of 0 or less (or NaN) takes the
 * first token, with probability 1.  Logits of -inf or NaN are no tokens, +inf
 * counts as the type's largest finite number.  A row without tokens gets index
 * -1 and probability 0.
 * temperature, top_p, min_p (fp32) and top_k (int32), each [n_rows], may be
 * NULL: 1, and no cut (nor does a NaN of top_p or min_p cut).  u below 0 or NaN
 * counts as 0, from 1 on as just below.  Weights are held as whole multiples of 2^-s, s = 50 up to
 * 4096 tokens and one less for each doubling of the vocabulary from there, and
 * summed as whole numbers: the same bit for bit from run to run, and no choice
 * falls otherwise than in 64 bits unless it lies within that rounding.  At
 * temperatures below 2^-100 only the tokens of the largest logit weigh
 * anything. */
rfpx_status rfpx_sample(const void *logits_dev, long long stride, int xtype, int n_rows, int vocab,
                        const float *u_dev, const float *temperature_dev,
                        const int32_t *top_k_dev, const float *top_p_dev, const float *min_p_dev,
                        int32_t *tokens_dev, float *probs_dev, void *ws_dev, size_t ws_bytes,
                        void *stream);

/* Follow every sequence's tree from column 0: the next column is the first
 * one whose parent this is and whose token (tokens_dev [n_rows]) is the one
 * drawn at its parent (drawn_dev [n_rows], as rfpx_sample gives it; a negative
 * one confirms nothing), as far as there is one and path_cols columns allow.
 *   path[b][..]  the columns, ascending, then -1   (int32 [n_seqs][path_cols])
 *   counts[b]    how many                          (int32 [n_seqs])
 *   next[b]      the token drawn at the last       (int32 [n_seqs])
 *   lens_out[b]  lens[b] - n + counts[b], 0 or more  (int32 [n_seqs], or NULL)
 * A sequence without columns: no path, count 0, next -1.  lens_out may be
 * b->lens itself, but not where rfpx_kv_commit follows with the same batch: that
 * needs the lengths of the step. */
rfpx_status rfpx_tree_accept(const rfpx_kv_batch *b, int n_rows, const int32_t *parents_dev,
                             const int32_t *tokens_dev, const int32_t *drawn_dev, int path_cols,
                             int32_t *path_dev, int32_t *counts_dev, int32_t *next_dev,
                             int32_t *lens_out_dev, void *stream);

/* For every sequence and kv head, move slot lens[b] - n + path[b][i] to slot
 * lens[b] - n + i, for i < counts[b]: keys and values, and of acc_dev and
 * pos_dev (fp32 and int32 [n_seqs][n_kv_heads][pages_per_seq * page_tokens],
 * each or both NULL) the same slots.  lens and starts are those of the step.
 * The path is ascending, so that an entry is its own index or more; an entry
 * below its index or that is no column of the step is passed over, and so is one
 * that would move to a negative slot.  A move from or to a slot without a page in
 * the pool carries acc and pos only.  Sequences must not share the pages of the
 * step's columns. */
rfpx_status rfpx_kv_commit(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int path_cols,
                           const int32_t *path_dev, const int32_t *counts_dev, float *acc_dev,
                           int32_t *pos_dev, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* RFPX_VERIFY_H */

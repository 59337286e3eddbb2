/*
 * rfpx_attn.h -- C ABI of librfpx, attention: the step between a layer's
 * packed qkv projection (rfpx_dense_forward) and its output projection, over
 * a paged key/value cache held in RFPX_FP4 blocks.
 *
 *   rfpx_qk_norm_rope   RMS norm of every query and key head, and the
 *                       rotation by position, in one pass
 *   rfpx_kv_append      keys and values quantized into the cache
 *   rfpx_kv_unpack      what the cache holds, as fp32 or bf16 values
 *   rfpx_attn_forward   attention of new columns over the cache
 *   rfpx_attn_weights   the attention weight every cached token has gathered
 *   rfpx_kv_evict       tokens of little weight leave the cache
 *
 * The conventions of rfpx.h hold: device pointers of the current device end
 * in _dev, everything is checked on the host before anything is enqueued,
 * nothing is allocated, kept between calls or synchronized, and a non-zero
 * rfpx_status leaves a text in rfpx_last_error().
 *
 * ------------------------------------------------------------- the cache
 * A token's D = head_dim values of one kv head are D/32 FP4 blocks of 32
 * (w_j = (code_j - 7.5) * 2^(e-127), rfpx.h), 4.25 bits a value.  Pages of
 * page_tokens tokens lie in one pool.  A page holds, for every kv head in
 * turn, a slab of page_tokens * D * 17/16 bytes:
 *   keys    [token][octet of a block: 4][block: D/32][4 bytes]
 *   scales  [token][block]                        (e, one byte)
 *   values  [token/4][byte of a block: 16][pair of the four tokens: 2]
 *           [block/2][token & 1][block & 1]       (one byte)
 *   scales  [token][block]
 * which is a permutation of the canonical blocks' bytes: a lane of the
 * attention kernels reads its operand of a matrix instruction as it stands.
 *
 * Slot s of sequence b lies in page page_table[b][s / page_tokens], at token
 * s % page_tokens.  Keys are stored rotated, so the order of the slots
 * carries no meaning beyond "appended before".  A page number outside
 * [0, n_pages) is no memory: appends to it are dropped, and attention takes
 * its slots as not held.
 *
 * ------------------------------------------------------------- the batch
 * A step brings starts[b+1] - starts[b] new columns (rows starts[b] ..
 * starts[b+1]-1 of q, k, v and out) to sequence b, which holds lens[b] slots
 * with them: column i of n sits in slot lens[b] - n + i and attends to slots
 * 0 .. lens[b] - n + i.  A column whose slot is negative is not appended and
 * sees nothing.  starts is ascending from 0 or more; rows at or behind
 * starts[n_seqs], and at or behind n_rows, are neither read nor written.
 * lens past pages_per_seq * page_tokens counts as that.  Both arrays and the
 * page table are device data that each call reads, so that a captured graph
 * is replayed on other lengths; max_cols and max_len are what a launch is
 * planned for (a longer sequence is computed as well, only less evenly).
 */
#ifndef RFPX_ATTN_H
#define RFPX_ATTN_H

#include "rfpx.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RFPX_HEADS_MAX 1024  /* query heads, and kv heads */
#define RFPX_ROWS_MAX (1 << 20)
#define RFPX_SEQS_MAX 65535

typedef struct {
  int n_kv_heads;    /* 1..RFPX_HEADS_MAX */
  int head_dim;      /* 64, 128 or 256 */
  int page_tokens;   /* 32, 64, 128 or 256 */
  int n_pages;       /* pages of the pool, 1 or more */
  uint8_t *pool;     /* device, 256-byte aligned */
  size_t pool_bytes; /* at least rfpx_kv_pool_bytes() of the above */
} rfpx_kv_cache;

typedef struct {
  int n_seqs;                /* 1..RFPX_SEQS_MAX */
  int pages_per_seq;         /* row length of page_table, 1 or more; up to
                                2^30 tokens of pages */
  int max_cols;              /* most columns of a sequence in this step, 0.. */
  int max_len;               /* largest of lens, 0.. */
  const int32_t *page_table; /* device, [n_seqs][pages_per_seq] */
  const int32_t *lens;       /* device, [n_seqs] */
  const int32_t *starts;     /* device, [n_seqs + 1] */
} rfpx_kv_batch;

/* Pairs of one head's first `dim` values that a rotation turns. */
enum { RFPX_ROPE_HALF = 0,   /* i and i + dim/2 */
       RFPX_ROPE_PAIRS = 1   /* 2i and 2i + 1 */ };

typedef struct {
  int dim;                     /* rotated values, even, 0..head_dim; 0: none */
  int style;                   /* RFPX_ROPE_HALF or RFPX_ROPE_PAIRS */
  const double *inv_freq_host; /* host, [dim/2], radians a position; read
                                  before the call returns */
} rfpx_rope;

/* Bytes of a pool; 0 for an unsupported shape. */
size_t rfpx_kv_pool_bytes(int n_kv_heads, int head_dim, int page_tokens, int n_pages);

/* For every row and head of q [n_rows][n_heads][head_dim] and k [n_rows]
 * [n_kv_heads][head_dim] (fp32 or bf16 per xtype; rows q_stride and k_stride
 * elements apart, heads adjacent):
 *   z = x / sqrt(mean(x^2) + eps) * weight        (weight NULL: z = x)
 *   (z_a, z_b) -> (z_a cos t - z_b sin t, z_a sin t + z_b cos t)
 * for the pairs of rope, t = positions[row] * inv_freq, the angle reduced in
 * 64 bits (rope NULL: none).  All in fp32 (the sum of the squares too: values
 * past 2^60 are out of its range), rounded once into q_out and k_out
 * (fp32 or bf16 per otype), which may be q and k themselves with the same
 * stride and type.  A row of negative position is padding: left as it was.
 * q or k may be absent (NULL with 0 heads).  head_dim 64, 128 or 256;
 * pointers 16-byte aligned and strides a multiple of 16 bytes. */
rfpx_status rfpx_qk_norm_rope(const void *q_dev, long long q_stride, int n_heads,
                              const void *k_dev, long long k_stride, int n_kv_heads,
                              int head_dim, int xtype, int n_rows,
                              const int32_t *positions_dev, const float *q_weight_dev,
                              const float *k_weight_dev, float eps, const rfpx_rope *rope,
                              void *q_out_dev, long long q_out_stride, void *k_out_dev,
                              long long k_out_stride, int otype, void *stream);

/* Quantize the step's k and v ([n_rows][n_kv_heads][head_dim], fp32 or bf16)
 * into their slots by rfpx_pack's FP4 rule, bit for bit.  A block with a
 * value that is not finite is stored as e = 255: it reads as NaN.
 * pos_dev and acc_dev (each NULL or [n_seqs][n_kv_heads][pages_per_seq *
 * page_tokens]) get positions_dev[row] and 0 at the slot of every kv head:
 * what rfpx_kv_evict and rfpx_attn_weights keep of a token.  Two rows must
 * not share a slot.  Alignment as for rfpx_qk_norm_rope. */
rfpx_status rfpx_kv_append(const rfpx_kv_cache *c, const rfpx_kv_batch *b, const void *k_dev,
                           long long k_stride, const void *v_dev, long long v_stride, int xtype,
                           int n_rows, const int32_t *positions_dev, int32_t *pos_dev,
                           float *acc_dev, void *stream);

/* The values that the cache holds for the step's columns, k_dev and v_dev
 * [n_rows][n_kv_heads][head_dim] (contiguous; fp32 or bf16 per otype, exact
 * in both).  With as many columns as slots it reads a whole sequence.  Rows
 * without a slot or a page are left as they were. */
rfpx_status rfpx_kv_unpack(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int n_rows,
                           void *k_dev, void *v_dev, int otype, void *stream);

/* Workspace of rfpx_attn_forward; 0 if unsupported.  256-byte aligned, no
 * initialization needed, scratch between calls.  It depends on n_heads,
 * n_rows and the batch's sizes, not on device data. */
size_t rfpx_attn_workspace_bytes(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int n_heads,
                                 int n_rows);

/* For every column and query head (head h reads kv head h / (n_heads /
 * n_kv_heads)), over the slots that the column sees:
 *   s = scale * q . k,   out = sum softmax(s) v,   lse = log sum exp(s)
 * q and out [n_rows][n_heads][head_dim], fp32 or bf16 per xtype, rows
 * q_stride and out_stride elements apart; lse_dev NULL or fp32 [n_rows]
 * [n_heads].  A column that sees nothing gets out = 0, lse = -inf.  The
 * cache's values enter the products exactly.  bf16 q enters as it is, and its
 * softmax numerators rounded to bf16 (2^-8 of each at most); they are divided
 * by the sum of the rounded ones, or in plans of many rows of the unrounded
 * ones, so that out differs within that bound from plan to plan.  fp32 q and
 * its numerators enter as three bf16 terms, 24 bits: what is lost is lost in
 * the fp32 sums, of terms up to four times their result.  Sums and statistics
 * are fp32, in a fixed order: out is the same bit for bit from run to run (of
 * one plan: max_cols and max_len decide how a sequence is split).  Scores may
 * be of any finite size.  scale > 0, below 1e30.  out may not overlap q. */
rfpx_status rfpx_attn_forward(const rfpx_kv_cache *c, const rfpx_kv_batch *b, const void *q_dev,
                              long long q_stride, int xtype, int n_heads, int n_rows, float scale,
                              void *out_dev, long long out_stride, float *lse_dev, void *ws_dev,
                              size_t ws_bytes, void *stream);

/* acc_out[b][kv head][slot] = decay * acc[..] + sum of exp(s - lse) over the
 * step's columns that see the slot and the query heads of the kv head, for
 * the slots below lens[b]; others are left as they were.  acc and acc_out
 * [n_seqs][n_kv_heads][pages_per_seq * page_tokens] fp32, may be the same.
 * q, scale and lse as rfpx_attn_forward was given and gave them.  lse is an
 * fp32 number: a weight is off by about 2^-22 |lse| of itself, and from |lse|
 * = 2^20 on says little.  Sums in a fixed order. */
rfpx_status rfpx_attn_weights(const rfpx_kv_cache *c, const rfpx_kv_batch *b, const void *q_dev,
                              long long q_stride, int xtype, int n_heads, int n_rows, float scale,
                              const float *lse_dev, float decay, const float *acc_dev,
                              float *acc_out_dev, void *stream);

/* Workspace of rfpx_kv_evict; 0 if unsupported. */
size_t rfpx_kv_evict_workspace_bytes(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int keep);

/* Cut every sequence longer than keep to keep slots (starts is not read).
 * For each kv head by itself: slots of position above (largest position) -
 * recent are kept first, then those of largest acc (NaN below everything),
 * ties to the lower slot.  The kept slots at or behind keep, in ascending
 * order, move into the slots before it that are not kept, in ascending
 * order: keys, values, acc and pos with them; every other kept slot stays
 * where it is.  lens_out[b] = min(lens[b], keep); acc_out and pos_out get
 * the slots below it.  acc_out, pos_out and lens_out may be acc, pos and
 * b->lens themselves (and overlap them no other way).  0 <= recent, 1 <= keep.
 * Sequences must not share pages, and every slot below lens[b] must have its
 * page in the pool: the choice looks at acc and pos alone.  Of a sequence that
 * breaks this nothing outside the pool is read or written and others are not
 * touched, but its moves from or to such a page carry acc and pos only, keys
 * and values stay, and its slots no longer belong together. */
rfpx_status rfpx_kv_evict(const rfpx_kv_cache *c, const rfpx_kv_batch *b, int keep, int recent,
                          const float *acc_dev, const int32_t *pos_dev, float *acc_out_dev,
                          int32_t *pos_out_dev, int32_t *lens_out_dev, void *ws_dev,
                          size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* RFPX_ATTN_H */

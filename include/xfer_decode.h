/*
 * xfer_decode.h - the decode-step calls of libxfer, for AMD Instinct MI355X
 * (gfx950): what a decode worker computes around the transfers of xfer.h.
 *
 *   xfer_qkv_rope_store  norms of queries and keys for each head, the
 *                        position rotation, and the new keys and values
 *                        written into a paged cache
 *   xfer_attn_paged      attention of one new token of every request over
 *                        such a cache, the whole of it or a window and the
 *                        first tokens
 *   xfer_sample_merge    sampling with temperature, top-k, top-p and min-p
 *                        from logits in two column shards, beside
 *                        xfer_argmax_merge
 *
 * The caches are the ones that xfer_gather_runs, xfer_scatter_runs and
 * xfer_paged_copy move.  All conventions of xfer.h hold (host checks first,
 * hot calls only enqueue on `stream`, the caller owns every buffer, results
 * are deterministic, pointers belong to the device current on the calling
 * thread, empty work is XFER_OK with nothing enqueued) with one difference:
 * these calls compute in binary32 (or wider where stated), so their results
 * are rounded values of the formulas below, the same bits on every call with
 * the same arguments and inputs.
 */
#ifndef XFER_DECODE_H
#define XFER_DECODE_H

#include "xfer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------- the paged cache */

/* How a cache holds its elements. */
enum {
  XFER_KV_BF16 = 0, /* BF16 bit patterns                                   */
  XFER_KV_E4M3 = 1  /* 8-bit floats (4 exponent bits, 3 mantissa bits, no
                       infinities, 448 the largest), each standing for its
                       value times the head's scale                        */
};

/*
 * A paged cache of keys and values.  Element d of head h of slot s of page p
 * of the keys is at byte
 *   k + p * page_stride + s * token_stride + h * head_stride + d * (element bytes)
 * and the same of the values at v.  So pages may hold whole tokens
 * ([slot][head][dim]) or one block per head ([head][slot][dim]), and keys
 * and values may alternate in one buffer.
 */
typedef struct {
  void *k, *v;             /* (device) 16-byte aligned                       */
  const float *k_scale;    /* (device) F32[kv_heads]; NULL: all 1; XFER_KV_E4M3 only */
  const float *v_scale;    /* the same for the values                        */
  uint64_t page_stride;    /* bytes, multiples of 16                         */
  uint64_t token_stride;
  uint64_t head_stride;
  uint32_t n_pages;
  uint32_t page_tokens;    /* slots in a page: a power of two up to 65,536   */
  uint32_t kv_heads;
  uint32_t head_dim;       /* 64, 128 or 256                                 */
  int32_t kind;            /* XFER_KV_*                                      */
  uint32_t reserved;       /* 0                                              */
} xfer_kv_cache;

/*
 * The checks that every call makes of a cache: XFER_E_INVAL for a NULL cache,
 * NULL or misaligned k or v, a stride that is not a multiple of 16,
 * n_pages, page_tokens or kv_heads 0, page_tokens not a power of two, an
 * unknown kind, scales with XFER_KV_BF16, misaligned scales (4 bytes),
 * reserved not 0, or an extent that passes 2^47 bytes; XFER_E_UNSUPPORTED for another head_dim or page_tokens
 * above 65,536.
 */

/* ------------------------------------ norms, rotation and the cache's rows */

enum { XFER_ROPE_HALVES = 0, XFER_ROPE_PAIRS = 1 };

/* The position rotation. */
typedef struct {
  const float *cos_sin;     /* (device) F32[max_pos][rot_dim]: row p holds the
                               rot_dim / 2 cosines, then the sines, of position
                               p; 16-byte aligned; may be NULL if rot_dim is 0 */
  const int32_t *positions; /* (device) one per token; may be NULL if rot_dim is 0 */
  uint32_t max_pos;
  uint32_t rot_dim;         /* dims of a head that are rotated: a multiple of 8
                               up to head_dim, 0 for none                    */
  int32_t style;            /* XFER_ROPE_HALVES: dims i and i + rot_dim / 2
                               form a pair; XFER_ROPE_PAIRS: 2i and 2i + 1   */
  uint32_t reserved;        /* 0                                             */
} xfer_rope;

/* The projections of a batch of tokens: row t of q holds q_heads heads of
 * head_dim BF16 elements one after the other, rows of k and v kv_heads.  The
 * three may be slices of one buffer. */
typedef struct {
  const uint16_t *q, *k, *v;        /* (device) 16-byte aligned               */
  uint64_t q_ld, k_ld, v_ld;        /* elements between rows, multiples of 8  */
  const uint16_t *q_weight;         /* (device) BF16[head_dim], 16-byte aligned;
                                       NULL: queries are not normalised       */
  const uint16_t *k_weight;         /* the same for the keys                  */
  uint32_t tokens;
  uint32_t q_heads;                 /* any count, 0 for keys and values alone */
  float eps;                        /* finite, >= 0                           */
  uint32_t reserved;                /* 0                                      */
} xfer_qkv;

/*
 * xfer_qkv_rope_store - for every token t and every head of q and k:
 *   y_d  = x_d * 1 / sqrt(mean_d(x_d^2) + eps) * weight_d   (x_d if no weight)
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)  for each pair (a, b)
 * with the cosines and sines of the token's position.  The queries go to
 * q_out (BF16, row t at q_out + t * q_out_ld, heads one after the other), the
 * keys to slot slots[t] of the cache, and the values, unchanged, to the same
 * slot.  Everything is computed in binary32 (the sum of a head's squares too,
 * which has to stay within it: |x| below 2^59 does) and rounded once, to
 * nearest even: to BF16, or to E4M3 of (value / the head's scale) limited to
 * +-448.  NaN stays NaN, though not always the same one.
 *
 *   slots  (device) int64[tokens]: page * page_tokens + slot.  A token whose
 *          slot is negative, or not below n_pages * page_tokens, is not
 *          stored (its queries are written all the same).  The slots that are
 *          stored to must be distinct: which token's bytes remain in a slot
 *          named twice is unspecified.
 *   q_out  may be q itself with the same ld (computed in place); NULL is
 *          allowed if q_heads is 0.
 *
 * A token whose position is not in [0, max_pos) gets NaN queries and is not
 * stored.  No byte of the cache outside the named slots is written.
 *
 * Errors: those of the cache; XFER_E_OVERLAP if two slots of the cache share
 * bytes, of keys, of values or one of each; XFER_E_INVAL for NULL or
 * misaligned pointers (k, v, q and q_out where there are heads; slots, 8
 * bytes), lds that are not multiples of 8 or
 * smaller than a row, a q_out row that overlaps a row of q, k or v (except in
 * place), another input or the cache, an input overlapping the cache, eps negative or not
 * finite, rot_dim not a multiple of 8 or above head_dim, a rotation with NULL
 * or misaligned table, NULL or misaligned positions (4 bytes) or max_pos 0, an unknown style, or a
 * reserved field that is not 0; XFER_E_UNSUPPORTED if the call needs more
 * than 2^24 - 1 workgroups (about one for 16 heads of a token).
 */
XFER_API int xfer_qkv_rope_store(const xfer_kv_cache *cache, const xfer_qkv *in, const xfer_rope *rope,
                                 const int64_t *slots, uint16_t *q_out, uint64_t q_out_ld, hipStream_t stream);

/* ------------------------------------------- attention of one new token */

/*
 * The requests of a batch: row r's token j (its position in the request,
 * from 0) lies in slot j mod page_tokens of page
 * page_table[r * table_ld + j / page_tokens].
 */
typedef struct {
  const uint32_t *page_table; /* (device) rows of at least
                                 ceil(max_len / page_tokens) page numbers     */
  const uint32_t *lens;       /* (device) tokens in the cache of each row, the
                                 new one among them; above max_len: max_len   */
  uint64_t table_ld;          /* page numbers between rows                    */
  uint32_t rows;
  uint32_t max_len;           /* the longest row (an upper bound will do, but
                                 the work is cut up for rows of this length)  */
  uint32_t window;            /* 0: every token is visible; else the last
                                 `window` tokens and the first `sinks`        */
  uint32_t sinks;             /* 0 if window is 0                             */
} xfer_paged_batch;

/*
 * xfer_attn_paged - for every row r and query head h, with kv head
 * g = h / (q_heads / kv_heads) and the row's visible tokens j:
 *   s_j = scale * q[r][h] . k_j        (k_j times k_scale[g] if there is one)
 *   out[r][h] = sum_j exp(s_j - max s) v_j / sum_j exp(s_j - max s)
 *                                      (v_j times v_scale[g])
 * A row with no visible token (length 0, or holes alone) gets zeros, and so
 * does a head whose scores are all -inf.  A page
 * number that is not below n_pages is a hole: its tokens are not visible and
 * nothing is read for them.  What pages hold past a row's length, and tokens
 * outside the window, has no influence, NaN and infinities included.
 *
 * Among a row's visible tokens, an infinite value makes its dim of every head
 * of its kv head that infinity, however small its weight; a NaN, or infinities
 * of both signs, make it NaN.  A score of NaN or +inf makes its head NaN.
 * Neither reaches another dim, head or row.  Finite inputs give finite results
 * where q . k_j, the score and the sum of a dim's values, each times up to 2^8,
 * stay within binary32.
 *
 * Several new tokens of one request are rows of their own, with the same
 * page numbers and increasing lengths.
 *
 * Scores, maxima, sums and the weighted sum are held in binary32; a weight
 * is split into BF16 numbers for the product with v, which keep it to 2^-17
 * of itself (two numbers, for XFER_OUT_BF16) or, from 2^-100 on, exactly
 * (three, for XFER_OUT_F32).  The result is rounded once, to nearest even, for
 * XFER_OUT_BF16.
 *
 *   q         (device) BF16 bit patterns, row r at q + r * q_ld, q_heads
 *             heads of head_dim one after the other; 16-byte aligned, q_ld a
 *             multiple of 8.
 *   out       (device) the same of BF16 or F32 (out_mode XFER_OUT_*), rows
 *             out_ld elements apart (a multiple of 8).
 *   workspace (device) at least xfer_attn_workspace_bytes() bytes, 16-byte
 *             aligned, any contents: the partial results of rows that are cut
 *             up.  May be NULL if that is 0.  Calls that may run concurrently
 *             must use different workspaces.
 *
 * Errors: those of the cache; XFER_E_INVAL for NULL or misaligned pointers
 * (page_table and lens 4 bytes), q_heads not a positive multiple of kv_heads,
 * a scale that is not finite, sinks without a window, max_len 0 or above
 * 2^31 - 1, a table_ld below ceil(max_len / page_tokens) (rows > 1), lds that
 * are not multiples of 8 or smaller than a row, an unknown out_mode, a small
 * workspace, or an output or workspace that overlaps q, the cache, its scales,
 * the table, the lengths or one another; XFER_E_UNSUPPORTED for more than 2^24 - 1
 * workgroups.
 *
 * xfer_attn_workspace_bytes - the bytes that such a call needs (0 also for
 * sizes and caches that xfer_attn_paged refuses).  They depend on the sizes and
 * strides alone, not on pointers.
 */
XFER_API size_t xfer_attn_workspace_bytes(const xfer_kv_cache *cache, const xfer_paged_batch *batch,
                                          uint32_t q_heads);
XFER_API int xfer_attn_paged(const xfer_kv_cache *cache, const xfer_paged_batch *batch, const uint16_t *q,
                             uint64_t q_ld, uint32_t q_heads, float scale, void *out, uint64_t out_ld, int out_mode,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);

/* --------------------------------------------------------------- sampling */

/* One row's settings. */
typedef struct {
  float temperature; /* logits are divided by it; not above 0, or NaN: the
                        first element of the row's order is taken (greedy)    */
  uint32_t top_k;    /* keep the first top_k elements; 0: all                 */
  float top_p;       /* keep the shortest prefix of those whose weights sum to
                        top_p of theirs, one element at least; 1 or more, or
                        NaN: all                                              */
  float min_p;       /* of those, keep elements whose weight is at least min_p
                        times the largest; above 1 counts as 1; NaN: all      */
} xfer_sample_params; /* 16 bytes */

typedef struct {
  float prob;  /* the taken element's probability among the kept ones */
  int32_t idx; /* its global id, -1 if the row has nothing to take    */
} xfer_sampled; /* 8 bytes */

/*
 * xfer_sample_merge - one element of every row of a block of logit rows split
 * by columns between two ranks (the shards of xfer_argmax_merge), drawn by a
 * given number u in [0, 1).
 *
 * Row order: as xfer_argmax_merge, larger value first (numeric, -0 == +0),
 * then the lower global id.  With l_i in that order and T the temperature,
 * w_i = exp((l_i - l_0) / T) (an element equal to l_0 has weight 1, infinite
 * ones included).  Elements that are -inf (masked) or NaN are never taken and
 * count nowhere.  top_k, then top_p, then min_p each keep a prefix of the
 * order.  With Z the kept weights' sum, the taken element is the first whose
 * running sum of weights exceeds u * Z (the last kept one if rounding leaves
 * none; u below 0 or NaN counts as 0), and prob = w / Z.  Greedy rows keep
 * one element, so prob is 1.
 *
 * Weights and their sums are computed in binary64.  A BF16 logit has at most
 * 65,536 values, so a row is counted by value and equal logits share one
 * exponential.
 *
 *   params     (device) xfer_sample_params[rows], 16-byte aligned.
 *   u          (device) F32[rows].
 *   out        (device) xfer_sampled[rows], 16-byte aligned.
 *   workspace  (device) at least xfer_sample_workspace_bytes(rows, s0->ncols,
 *              s1->ncols) bytes, 16-byte aligned, any contents.  Calls that
 *              may run concurrently must use different workspaces.
 *
 * Errors: XFER_E_INVAL for NULL or misaligned pointers (ptr and ld * 2 must
 * be multiples of 16, u of 4), different row counts, ncols == 0, shards whose
 * id ranges overlap, col_offset + ncols > 2^31, a small workspace, or an
 * output or workspace overlapping an input or one another;
 * XFER_E_UNSUPPORTED for a shard wider than 2,097,152 columns or more than
 * 2^24 - 1 workgroups (one for a row, and one for each 16,384 columns or part
 * of a shard where a row has more than 32,768).
 */
XFER_API size_t xfer_sample_workspace_bytes(uint32_t rows, uint32_t ncols0, uint32_t ncols1);
XFER_API int xfer_sample_merge(const xfer_shard *s0, const xfer_shard *s1, const xfer_sample_params *params,
                               const float *u, void *out, void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* XFER_DECODE_H */

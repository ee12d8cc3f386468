/*
 * qpn_kv.h -- C ABI of the operators of a speculative round that stand around
 * the packed-weight products of qpn.h: page tables, the cache append with
 * query/key norms and rotation, attention over an 8-bit paged KV cache, the
 * verification of sampled drafts, and the log probabilities that a server answers
 * with.  MI355X (gfx950).  The operators of a 4-bit cache: qpn_kv4.h.
 *
 * One round on the device, without a host read:
 *   qpn_kv_plan_round      rows and lengths of the requests -> page tables,
 *                          row_start, slots, positions
 *   (QKV product)          qpn_gemm_* / qpn_gemm_prefill_*
 *   qpn_kv_rope_append     norm and rotate queries and keys, keys and values
 *                          into the cache
 *   qpn_kv_attention       the rows against the cache
 *   (O, gate/up, down, lm_head products)
 *   qpn_kv_verify_sampled  accepted drafts and the next token
 *   qpn_kv_logprobs        log probabilities of tokens, entropy, alternatives
 *
 * The cache of one layer.  Pages of QPN_KV_PAGE = 64 tokens; per page and KV
 * head the keys and the values are one block each of 64 * dim E4M3 codes
 * (OCP "FN") with one FP32 scale (a value is its code times the scale):
 *   keys    [dim / 16][64][16]: dimension 16 c + e of token t at (c, t, e);
 *   values  [dim][4][4][4]:     dimension d of token 16 t + 4 g + r at
 *                               (d, g, t, r).
 * Both orders are what one 16-byte load per lane hands the 16x16x32 f16 MFMA,
 * each load instruction covering whole 128-byte lines: the 16 dimensions of
 * a token's key for the scores, and of values the 16 tokens whose weights a
 * lane holds after the scores (its four accumulator rows of four tiles).
 * Blocks lie at (page * heads + head) * 64 * dim, scales at page * heads + head.
 *
 * Conventions as in qpn.h: device pointers on the current device unless noted,
 * FP16 as uint16_t bit patterns, all work enqueued on `stream`, no
 * allocation, no synchronisation, argument checks on the host before anything
 * is enqueued, QPN_ERR_* codes.  What a kernel reads on the device (lengths,
 * page and slot numbers, token ids) is bounds-checked there: a bad value gives
 * the documented result (a skipped row, NaN, -1), never an access out of range.
 * Rows of the requests lie one after another: request r has rows
 * row_start[r] .. row_start[r + 1] - 1.
 *
 * Scratch.  Attention, verification and log probabilities take device scratch of their own
 * (16-byte aligned; not the workspace of qpn.h): its first
 * QPN_KV_SCRATCH_ZEROED bytes must be zero before its first use and every call
 * leaves them zero; the rest may hold anything.  Calls that share a scratch
 * must not overlap.
 */
#ifndef QPN_KV_H
#define QPN_KV_H

#include "qpn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QPN_KV_PAGE 64
#define QPN_KV_SCRATCH_ZEROED 65536

/* One layer's cache (a host struct of device pointers, read by the call). */
typedef struct qpn_kv_cache {
  void *k;        /* pages * heads blocks of 64 * dim codes, 16-byte aligned */
  void *v;        /* as k */
  float *k_scale; /* [pages, heads] */
  float *v_scale; /* [pages, heads] */
  int64_t pages;  /* 1 .. 2^25 - 1 */
  int32_t heads;  /* KV heads, 1 .. 1024 */
  int32_t dim;    /* 64, 128 or 256 */
} qpn_kv_cache;

/* The tables of a round from the requests' lengths.  before[r]: tokens of
 * request r already in the cache; rows[r]: rows it brings; held[r]: pages
 * already in its table row (at least ceil(before / 64)).  It needs
 * n = ceil((before + rows) / 64) pages and takes w = max(0, n - held) from the
 * end of the free list: the k-th page taken in the call (requests in order) is
 * free_pages[*free_count - 1 - k].  A request is well formed when before, rows
 * and held are not negative, held and n are at most table_width and before is
 * at most 64 * held; it is admitted when, over the well-formed requests up to
 * and including it, the sum of w is at most *free_count (clamped to 0 ..
 * free_capacity) and the sum of rows at most capacity.  One that is not
 * admitted gets no rows and no pages.
 * Written: seq_lens[r] = before + admitted rows (0 when not well formed);
 * row_start[requests + 1]; held_out[r]; *free_count_out; the new entries
 * table[r][held .. held + w); for every row of capacity its slot
 * page * 64 + offset and its position (slot -1, position 0 behind the last
 * row).  held_out may be held, free_count_out may be free_count.
 * 0 <= requests <= 4096, 0 <= capacity <= 2^20, table_width < 2^25.
 * One kernel of one workgroup. */
QPN_API int qpn_kv_plan_round(const int32_t *before, const int32_t *rows, const int32_t *held,
                              int requests, int32_t *table, int64_t table_stride, int table_width,
                              const int32_t *free_pages, int64_t free_capacity,
                              const int32_t *free_count, int capacity, int32_t *seq_lens,
                              int32_t *row_start, int32_t *held_out, int32_t *free_count_out,
                              int32_t *slots, int32_t *positions, void *stream);

/* Norms, rotation and cache append of one layer's QKV rows, in one launch.
 * qkv: [rows, (q_heads + 2 heads) * dim] FP16 with row stride qkv_stride
 * elements (a multiple of 8): queries, keys, values.  For a query or key x:
 *   n = x / sqrt(mean(x^2) + eps) * weight   (n = x when weight is NULL);
 *   over the first `rot` dimensions (a multiple of 16), with angle
 *   t_j = position * inv_freq[j], j < rot / 2:
 *   (a, b) -> (a cos t_j - b sin t_j, b cos t_j + a sin t_j) on the pair
 *   (j, j + rot / 2), or (2 j, 2 j + 1) when interleaved.
 * Queries go to q_out [rows, q_heads * dim] FP16 (row stride q_stride; q_out
 * may be qkv, with its stride).  Keys and values of a row with a slot in [0, 64 * pages) go to
 * the cache; other rows only write their queries.  Per page, head and kind:
 *   s = the smallest power of two with amax <= 448 s (at least 2^-60), amax
 *   over the finite new values; unless the page's first token (slot % 64 ==
 *   0) is among the new ones, s is at least the page's former scale, and if
 *   s grows the codes already there are rounded again to E4M3(code * old / s);
 *   new codes are E4M3(x / s), to nearest, ties to even, saturating, NaN to
 *   NaN.  Of two rows with one slot the later row counts.
 * Queries are computed in FP32, with angles reduced in FP64 and the hardware's
 * sine and cosine, which are off by up to 2^-20: before its rounding to FP16 a
 * rotated query is off by some 2^-19 of its pair's length.  Keys are computed
 * in FP64 up to their codes, so a key's code differs from the definition's only
 * where its value is within 3e-14 of its pair's length of a border between two
 * codes (position * inv_freq is exact for positions below 2^29 and rounded to
 * 64 bits above).  Codes of values, and of keys neither normed nor rotated, are
 * the definition's, for any scale that a page has.
 * A page is written by one workgroup, which looks through all slots for its
 * rows: the time of a call grows with rows times pages.
 * 0 <= rows <= 2^20, q_heads a multiple of the cache's heads (at most 64 each);
 * rows * (q_heads + heads) <= 2^30, rows * heads <= 2^25, eps >= 0.  Alignment:
 * qkv and q_out 16, weights 16, positions, slots 4. */
QPN_API int qpn_kv_rope_append(const qpn_kv_cache *cache, const uint16_t *qkv, int64_t qkv_stride,
                               int rows, int q_heads, const uint16_t *q_weight,
                               const uint16_t *k_weight, double eps, const float *inv_freq, int rot,
                               int interleaved, const int32_t *positions, const int32_t *slots,
                               uint16_t *q_out, int64_t q_stride, void *stream);

/* Bytes of scratch qpn_kv_attention wants for these sizes ((size_t)-1 for
 * sizes out of range).  With less (at least QPN_KV_SCRATCH_ZEROED, or none at
 * all) it runs with fewer pieces along the cache.  Pure host. */
QPN_API size_t qpn_kv_attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads,
                                              int dim, int table_width);

/* Attention of a round's rows over the cache.  Row i of request r (of n_r
 * rows) stands at position p = seq_lens[r] - n_r + i; with query head h and
 * KV head h / (q_heads / heads):
 *   y = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),
 *   over the tokens j <= p (and j > p - window when window > 0) of the pages
 *   table[r][j / 64].
 * q: [rows, q_heads * dim] FP16 (row stride q_stride, a multiple of 8), y the
 * same (row stride y_stride, a multiple of 4).  A row that sees no token gives
 * zeros; what stands in tokens a row does not see (NaN included) never reaches
 * it.  A page number outside the cache, or a page whose values' scale is
 * negative, infinite or NaN, gives NaN in the rows that see it, and
 * seq_lens[r] > 64 * table_width gives NaN in all rows of r.  Requests whose
 * row_start is out of order or past `rows` are skipped; rows of no request are
 * not written.  max_rows: the most rows of one request, a hint that the tile
 * is chosen by.
 * Scores, weights' sums and outputs are held in FP32.  For the second product
 * each weight, in units in which a row's largest is from 1 to 2^8, is rounded
 * to FP16: it is off by up to 2^-11 of itself, or 2^-25 where it is below
 * 2^-14 (the output's own rounding: 2^-11).  With many rows a weight carries
 * its page's value scale as a factor from 1 to 2^7 then, so it keeps at least
 * these bits; values whose scale is below 2^-40 count as zeros there.
 * scale > 0, window >= 0.
 * Deterministic.  0 <= rows <= 2^20, rows * q_heads <= 2^30, requests <= 4096. */
QPN_API int qpn_kv_attention(const qpn_kv_cache *cache, const uint16_t *q, int64_t q_stride,
                             uint16_t *y, int64_t y_stride, int q_heads, int rows, int requests,
                             int max_rows, const int32_t *row_start, const int32_t *seq_lens,
                             const int32_t *table, int64_t table_stride, int table_width,
                             float scale, int window, void *scratch, size_t scratch_bytes,
                             void *stream);

/* Bytes of scratch qpn_kv_verify_sampled needs ((size_t)-1 for sizes out of
 * range).  Pure host. */
QPN_API size_t qpn_kv_verify_scratch_bytes(int rows, int requests, int64_t n);

/* Verification of drafted tokens against the target's probabilities, from
 * given random numbers (speculative sampling).  Row i of a request holds the
 * target's logits after its token tokens[row]; tokens[row + 1] is the draft
 * for that place (rows but the request's last).  With
 *   p = softmax(inv_temperature * logits[row]),
 *   q = softmax(inv_temperature * draft_logits[row]), or, when draft_logits is
 *       NULL, all of it on the draft (a greedy drafter),
 * the draft d of a row is accepted when accept_u[row] * q(d) < p(d).  L is the
 * number of drafts before the first one refused.  next[r] is the smallest x
 * with sum_{y <= x} w(y) > sample_u[r] * sum w (the last x with w(x) > 0 if
 * there is none), w = max(p - q, 0) of row L, or w = p when L is the last row
 * or that difference is nowhere positive.  Written: accepted[r] = L, next[r],
 * accept_prob[row] = min(1, p(d) / q(d)) (0 for a request's last row).
 * A draft outside 0 .. n - 1 is refused with accept_prob 0.  A target row with
 * NaN or +inf, or nothing above -inf, refuses its draft (accept_prob NaN) and
 * gives next = -1; a draft row like that refuses it too, and next comes from
 * p.  A request without rows gives accepted 0, next -1.  All sums and
 * exponentials are FP64, the latter off by up to 1.1e-12 of themselves.
 * 1 <= n <= 2^24, rows <= 65535, inv_temperature > 0 and finite; strides in
 * elements.  One kernel for a greedy drafter, two for a
 * sampled one. */
QPN_API int qpn_kv_verify_sampled(const uint16_t *logits, int64_t logits_stride,
                                  const uint16_t *draft_logits, int64_t draft_stride,
                                  const int32_t *tokens, const int32_t *row_start, int rows,
                                  int requests, int64_t n, double inv_temperature,
                                  const float *accept_u, const float *sample_u, int32_t *accepted,
                                  int32_t *next, float *accept_prob, void *scratch,
                                  size_t scratch_bytes, void *stream);

#define QPN_KV_MAX_TOP 32

/* Bytes of scratch qpn_kv_logprobs needs ((size_t)-1 for sizes out of range).
 * Pure host. */
QPN_API size_t qpn_kv_logprobs_scratch_bytes(int rows, int64_t n);

/* Log probabilities.  With p = softmax(inv_temperature * logits[row]) over the n
 * tokens of a row:
 *   logprob[row] = log p(tokens[row]),   entropy[row] = - sum p log p,
 *   top_ids[row][0 .. top - 1] and top_logprobs: the `top` tokens of the largest
 *   logits in falling order, of equal ones (-0 and 0 are) the lowest index first,
 *   and their log p.
 * A token outside 0 .. n - 1 has the log probability NaN; a logit of -inf has the
 * probability 0 and the log probability -inf.  A row with NaN or +inf, or nothing above
 * -inf, gives NaN throughout and ids of -1.
 * Exponentials are FP32, off by up to 2^-23 (1 + |x|) of themselves for exp(x); their
 * sum is FP64 and held so that a token's probability near 1 keeps a relative precision
 * of its distance from 1; results are rounded to FP32.  The same call on rows that lie
 * alike (sizes, top, address modulo 16 bytes) gives the same bits; the order of the sums
 * depends on these.
 * 0 <= rows <= 65535, 1 <= n <= 2^24, 0 <= top <= min(n, QPN_KV_MAX_TOP) (top_ids and
 * top_logprobs may be NULL when 0), inv_temperature > 0 and finite.  logits need
 * no more than their 2-byte alignment.  One kernel.  With top > 0, rows that mask all but
 * a few tokens, or hold few different values, take up to eight times as long as rows
 * whose logits spread. */
QPN_API int qpn_kv_logprobs(const uint16_t *logits, int64_t logits_stride, const int32_t *tokens,
                            int rows, int64_t n, double inv_temperature, int top, float *logprob,
                            float *entropy, int32_t *top_ids, float *top_logprobs, void *scratch,
                            size_t scratch_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QPN_KV_H */

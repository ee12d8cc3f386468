/*
 * qpn_kv4.h -- C ABI of the 4-bit paged KV cache: the append with query/key norms
 * and rotation, reading tokens back, and attention.  It takes the place of the
 * 8-bit cache of qpn_kv.h in a round; page tables and verification are the same.
 * MI355X (gfx950).
 *
 * The cache of one layer.  Pages of QPN_KV_PAGE = 64 tokens.  Of every token and KV
 * head, each 16 dimensions are one group: E2M1 codes (OCP: 0, 0.5, 1, 1.5, 2, 3, 4,
 * 6 and a sign) with an E4M3 scale (OCP "FN", not negative); a value is
 * code * scale * unit, the unit one FP32 number per head for keys and one for
 * values, chosen by the caller (positive and finite; 6 * 448 * unit is the largest
 * value, and groups whose largest is below 6 * 2^-6 * unit have coarser scales).
 * 4.5 bits a value.  A page and KV head has one block each of codes (32 dim
 * bytes) and of scales (4 dim bytes) for keys and for values, at
 * (page * heads + head) times their size.  With G = dim / 64:
 *
 *   keys, token 16 t + c and dimension 16 (G g + i) + e (t, g < 4; c, e < 16; i < G):
 *     codes  [2 G][64][16]: the lane 16 g + c has 16 bytes in each of 2 G rows; as
 *            pairs of eight bytes, pair n = t G + i holds the codes e = 0 .. 15 (even
 *            e in the lower four bits): row n / 2, bytes 8 (n % 2) on;
 *     scales [64][4 G]: of lane 16 g + c, group n at n.
 *   values, token 16 t + 4 g + r and dimension 16 (G a + i) + 4 j + b (t, g, r, a, j,
 *   b < 4; i < G):
 *     codes  [2 G][64][16]: the lane 16 g + 4 a + b has 32 G bytes, 16 in each row;
 *            their half bytes (the lower one first) are (t, r, i, j) in this order;
 *     scales [G][16][16]: of row i, lane 4 g + a, token (t, r) at 4 t + r.
 *
 * These are the orders in which one 16-byte load per lane hands both products of the
 * attention their operands on the 16x16x32 f16 MFMA, with whole groups in a lane.  A
 * group's scale is its token's own, so an append touches nothing but the new tokens.
 *
 * Conventions, scratch and bounds checks as in qpn_kv.h.
 */
#ifndef QPN_KV4_H
#define QPN_KV4_H

#include "qpn_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One layer's cache (a host struct of device pointers, read by the call). */
typedef struct qpn_kv4_cache {
  void *k;             /* pages * heads blocks of 32 dim bytes, 16-byte aligned */
  void *v;             /* as k */
  void *k_scale;       /* pages * heads blocks of 4 dim bytes, 16-byte aligned */
  void *v_scale;       /* as k_scale */
  const float *k_unit; /* [heads] */
  const float *v_unit; /* [heads] */
  int64_t pages;       /* 1 .. 2^25 - 1 */
  int32_t heads;       /* KV heads, 1 .. 1024 */
  int32_t dim;         /* 64, 128 or 256 */
} qpn_kv4_cache;

/* Norms, rotation and cache append of one layer's QKV rows, in one launch: queries,
 * rows and slots as in qpn_kv_rope_append.  Keys and values of a row with a slot go
 * to the cache; per group of 16 dimensions x, with u the head's unit:
 *   s = E4M3(max |x| / (6 u)), to nearest, ties to even, saturating at 448;
 *   codes E2M1(x / (s u)), to nearest, ties to even, saturating at 6; zeros when s = 0.
 * A group with an infinity or a NaN, or of a head whose unit is not positive and
 * finite, gets the scale NaN (0x7F) and codes zero: it reads as NaN.  Of two rows
 * with one slot the later row counts.  Nothing else in the cache is written.
 * Values are quantised exactly as defined.  Keys are computed in FP64 up to their
 * scales and codes, which differ from the definition's only where a value is within
 * 3e-14 of its pair's length of a bound between two of them.
 * A row looks through the slots behind its own: calls of very many rows grow with
 * their square (1024 rows: 16 KB of slots at most for a wavefront).
 * Limits and alignment as in qpn_kv_rope_append. */
QPN_API int qpn_kv4_rope_append(const qpn_kv4_cache *cache, const uint16_t *qkv, int64_t qkv_stride,
                                int rows, int q_heads, const uint16_t *q_weight,
                                const uint16_t *k_weight, double eps, const float *inv_freq, int rot,
                                int interleaved, const int32_t *positions, const int32_t *slots,
                                uint16_t *q_out, int64_t q_stride, void *stream);

/* Tokens of the cache as FP16 rows: k_out and v_out [rows, heads * dim] (row strides
 * in elements, multiples of 8; 16-byte aligned) hold the keys and the values of the
 * tokens slots[0 .. rows - 1] (page * 64 + offset; in any order, the same one as often
 * as wanted), code * scale exact, times the unit in FP32, rounded to FP16.  A slot
 * outside [0, 64 * pages) gives zeros; a unit that is not positive and finite NaN.
 * 0 <= rows <= 2^20, rows * heads <= 2^25. */
QPN_API int qpn_kv4_read(const qpn_kv4_cache *cache, const int32_t *slots, int rows,
                         uint16_t *k_out, int64_t k_stride, uint16_t *v_out, int64_t v_stride,
                         void *stream);

/* Bytes of scratch qpn_kv4_attention wants, as qpn_kv_attention_scratch_bytes. */
QPN_API size_t qpn_kv4_attention_scratch_bytes(int requests, int max_rows, int q_heads, int heads,
                                               int dim, int table_width);

/* Attention of a round's rows over the cache: arguments, masks, rows and results for
 * bad input as in qpn_kv_attention, with the values of this cache.  A page number
 * outside the cache, a key group whose scale is NaN, or a unit that is not positive and
 * finite gives NaN in the rows that see it; a value group whose scale is NaN gives NaN
 * in its 16 dimensions of the rows that see it.
 * Scores (times log2 e), weights' sums and outputs are held in FP32: a row with a score
 * of 2^127 or more may be NaN.  Keys and values enter the products as code * scale, exact
 * in FP16.  For the second product each weight, in units in which a row's largest is from
 * 1 to 2^8, is rounded to FP16: it is off by up to 2^-11 of itself, or 2^-25 where it is
 * below 2^-14 (the output's own rounding: 2^-11).  Deterministic.
 * table_width is also the hint of the longest request, by which the work is split: with
 * several rows x query heads of a KV head and few requests, a table much wider than the
 * requests need costs about half as much again. */
QPN_API int qpn_kv4_attention(const qpn_kv4_cache *cache, const uint16_t *q, int64_t q_stride,
                              uint16_t *y, int64_t y_stride, int q_heads, int rows, int requests,
                              int max_rows, const int32_t *row_start, const int32_t *seq_lens,
                              const int32_t *table, int64_t table_stride, int table_width,
                              float scale, int window, void *scratch, size_t scratch_bytes,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QPN_KV4_H */

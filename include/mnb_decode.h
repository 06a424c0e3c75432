/*
 * mnb_decode.h -- the operators of a decoding step around the attention and behind the logits
 * that libmnb also exports: appending to a paged key/value cache held in MX FP4 (norms of
 * queries and keys for each head, rotation and quantisation in one pass), reading its rows
 * back, attention over it, and sampling.  One AMD Instinct MI355X (gfx950).
 *
 * Conventions are those of mnb_ops.h: device pointers (but the two structs, which are read on the
 * host), status codes, `stream`, the caller owns every buffer, nothing is synchronised,
 * arguments are validated before anything is enqueued, row distances in elements, an output
 * shares no byte with an input or another output but where said, workspaces need no
 * initialisation and hold nothing between calls.  Calls that may overlap in time use different
 * workspaces, and no call may write cache rows that another reads at the same time.
 */
#ifndef MNB_DECODE_H
#define MNB_DECODE_H

#include "mnb_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache: `pages` pages of `page_size` tokens for each of `kv_heads` heads of `head_dim`
 * elements, keys and values in MX FP4 along the head (blocks of 32).
 *   head_dim 64, 96, 128, 192 or 256; page_size a power of two from 16 to 65536;
 *   else MNB_ERR_UNSUPPORTED.
 * Page p starts at data + p * page_stride; page_stride is at least mnb_kv_page_bytes and a
 * multiple of 16, data 16-byte aligned.  Bytes of a page never written to may hold anything.
 *
 * Layout of a page: for each head, in bytes, with S = page_size, D = head_dim,
 *   key codes     [S][D / 2]           at 0             even index in the low nibble
 *   value codes   [S / 4][D / 8][4][4] at S D / 2       (group of 4 tokens, 8 elements, token, bytes)
 *   key scales    [S][D / 32]          at S D
 *   value scales  [S / 4][D / 32][4]   at S D + S D / 32
 */
typedef struct {
  void *data;
  int64_t page_stride;
  int pages, kv_heads, head_dim, page_size;
} mnb_kv_cache;

/*
 * The rows of a call: `rows` of them, of `batch` sequences.
 *   lengths [batch]    tokens of each sequence in the cache, the rows of the call counted
 *   starts [batch + 1] sequence b has the rows starts[b] .. starts[b + 1] - 1, n of them, its last
 *                      tokens: row starts[b] + i is at position lengths[b] - n + i.  starts[0] is 0 and
 *                      they do not fall.  NULL: one row for each sequence (rows == batch).
 *   pages [batch, width] (ldp elements between rows): position p lies in page pages[b][p / page_size]
 * All int32 on the device.  What only the device sees is checked there, without an access out of
 * bounds:
 *   - a row at a negative position (a sequence of length 0 that is given a row) has no
 *     position: its results are zeros and nothing is stored for it;
 *   - a position past width * page_size, or in a page whose number is not in [0, pages), stores nothing and
 *     its row becomes NaN; one past the rotation table's end stores NaN in its place (keys and values), and its
 *     row becomes NaN.  Attention gives NaN in rows that see such a position, and may in other rows of that sequence;
 *   - rows at or behind starts[batch] belong to no sequence and are left as they were.
 * Limits, past which a call is MNB_ERR_UNSUPPORTED: width * page_size 2^30, rows and batch below 2^22, heads 65536, rows * q_heads
 * 2^30, and attention's tiles of 16 or 32 rows of all key/value heads 2^23.
 */
typedef struct {
  const int32_t *pages;
  int64_t ldp;
  const int32_t *lengths, *starts;
  int batch, width, rows;
} mnb_kv_rows;

/* Bytes of a page of all heads; 0 where the sizes are not supported. */
size_t mnb_kv_page_bytes(int kv_heads, int head_dim, int page_size);

/*
 * For each row: queries q [rows, q_heads, head_dim] and keys k [rows, kv_heads, head_dim] are taken to
 *   h = x / sqrt(mean(x^2) + eps) * weight    over each head, where a weight [head_dim] is given,
 * then their first `rot` elements are rotated by row p of the table at position p, which holds
 * rot / 2 cosines and as many sines (FP32, [table_rows, rot]):
 *   (a, b) -> (a cos - b sin, b cos + a sin)   for the pairs (i, i + rot / 2), or
 *                                              (2 i, 2 i + 1) with `interleaved`.
 * q_out [rows, q_heads, head_dim] receives the queries (means in 64 bits, products in 32, one rounding to dtype);
 * keys, and values v as they are, go to the cache as by mnb_mx_quantize of the exact (64-bit) keys.
 * dtype fp16 or bf16 for q, k, v, weights and q_out.  rot a multiple of 16 up to head_dim, or 0 and no table.
 * q may be NULL with q_heads 0 (then q_out is not used); q_out may be q itself.
 * Tensors 16-byte aligned, as are their row distances in bytes; heads lie head_dim elements apart.
 * Two rows of a call at one position of one page leave either's bytes there.
 */
int mnb_kv_append(const mnb_kv_cache *cache, const mnb_kv_rows *rows, const void *q, int64_t ldq, int q_heads, const void *k,
                  int64_t ldk, const void *v, int64_t ldv, int dtype, const float *table, int table_rows, int rot,
                  int interleaved, const void *q_weight, const void *k_weight, float eps, void *q_out, int64_t ldo,
                  void *stream);

/* The cache's values at the rows' positions as k and v [rows, kv_heads, head_dim], rounded once to
 * `dtype` (any of the three); either may be NULL.  Aligned as above. */
int mnb_kv_read(const mnb_kv_cache *cache, const mnb_kv_rows *rows, void *k, int64_t ldk, void *v, int64_t ldv, int dtype,
                void *stream);

/*
 * y = softmax(scale q . k) v for each row and query head over the tokens that the row sees: those up to its own
 * position p and, where window > 0, behind p - window.  q_heads is a multiple of kv_heads; query
 * head h reads key/value head h / (q_heads / kv_heads).  A row that sees nothing is zeros.
 * q, y [rows, q_heads, head_dim] fp16 or bf16, aligned as above; y may be q itself.  Scores and sums are in
 * 32 bits; probabilities, keys and values enter the matrix instructions in q's type.  bf16 holds every
 * key and value exactly; fp16 in steps of 2^-24, values up to 65504, as fp16 data gives, and keys up to 2^31, more than a
 * norm, weights and a rotation make of fp16 data.  What is larger (appended in bf16, read with fp16 queries) becomes infinite.
 * NaN or infinities among tokens that a row does not see do not reach it.
 * workspace: at least mnb_kv_attention_workspace_bytes bytes, 16-byte aligned (NULL if that is 0).
 */
size_t mnb_kv_attention_workspace_bytes(const mnb_kv_cache *cache, const mnb_kv_rows *rows, int q_heads, int window);
int mnb_kv_attention(const mnb_kv_cache *cache, const mnb_kv_rows *rows, const void *q, int64_t ldq, int q_heads, int dtype,
                     float scale, int window, void *y, int64_t ldy, void *workspace, size_t ws_bytes, void *stream);

/* The kernels mnb_kv_attention would launch, as text (host only; of the structs only sizes and whether starts
 * is NULL are read). */
int mnb_kv_describe_route(const mnb_kv_cache *cache, const mnb_kv_rows *rows, int q_heads, int window, char *buf,
                          size_t buf_len);

/*
 * One token for each row of logits [M, V] (any of the three types, any element alignment, V <= 2^22) from
 * the number u[m] in [0, 1) (FP32).  With z = logits / temperature and p = softmax(z), tokens stay that are
 *   1. among the top_k largest (equal ones by the lower index; top_k <= 0: all),
 *   2. of these, renormalised, in the shortest run of largest ones whose sum reaches top_p
 *      (top_p >= 1: all; the largest always stays),
 *   3. of these, those with p >= min_p times the largest p (min_p <= 0: all; above 1 as 1),
 * and tokens[m] is the first, by index, with which the running sum of the p that stay exceeds u[m] times
 * their whole sum.  (u < 0 counts as 0, 1 and above as the largest number below 1.)
 * temperature 0: the largest logit, the lower index of equal ones.
 * A row that holds a NaN or +infinity or nothing but -infinity, a temperature that is negative, infinite or NaN, and a NaN in u, top_p
 * or min_p, have no distribution: tokens[m] = -1.
 * Each parameter is an array [M] (FP32, top_k int32) or, where that is NULL, the number beside it.
 * p and their sums are held in 64 bits as whole numbers of 2^-S of the largest p, S = min(46, 62 - ceil(log2 V)), so the choice
 * depends on no order of summation.  It is that of exact arithmetic unless u times the whole sum lies within (V / 4 + 1024) 2^-S
 * times the largest p of a border between tokens, or top_p times it within (5 V / 4 + 1024) 2^-S.
 */
int mnb_sample(const void *logits, int dtype, int M, int V, int64_t ldl, const float *u, const float *temperature,
               float temperature_all, const int32_t *top_k, int top_k_all, const float *top_p, float top_p_all,
               const float *min_p, float min_p_all, int64_t *tokens, void *stream);

/* Version of this header's calls (major * 100 + minor). */
int mnb_decode_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MNB_DECODE_H */

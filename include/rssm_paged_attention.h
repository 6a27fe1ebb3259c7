/*
 * rssm_paged_attention.h -- C ABI of the attention layers of a hybrid decoder
 * in librssm_materialize (MI355X, gfx950): append of a chunk of new tokens to
 * a paged key/value cache, and causal attention of those tokens over it, with
 * an optional sliding window and first tokens that stay visible.
 *
 * Sequence s has kv_len[s] tokens in the cache, the new ones included; its
 * q_s = seq_start[s+1] - seq_start[s] new tokens are the last of them, at
 * positions p = kv_len[s] - q_s .. kv_len[s] - 1.  Token j of the cache lies on
 * page page_table[s][j / page_size], row j mod page_size.  Head h of a query at
 * position p reads key/value head h / (num_q_heads / num_kv_heads):
 *     o = sum_j exp(scale q.k_j - m) v_j / sum_j exp(scale q.k_j - m)
 * over the visible tokens j <= p with (window == 0 or j > p - window or
 * j < sinks).  Tokens on a page outside [0, num_pages) are not visible.  A query that
 * sees nothing gets zeros (lse -infinity); one with a NaN among its visible scores gets NaN
 * (lse too).
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_PAGED_ATTENTION_H
#define RSSM_PAGED_ATTENTION_H

#include <stdint.h>

#include "rssm_materialize.h" /* dtype codes, rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side scalars (both entry points; the append ignores num_q_heads,
 * max_*, window, sinks, scale, the q, out and workspace fields, and takes
 * k_new and v_new with new_token_stride).
 *   num_seqs, num_tokens     sequences; rows of q / k_new / v_new (>= 0)
 *   num_q_heads, num_kv_heads  num_kv_heads divides num_q_heads
 *   head_dim                 64 or 128
 *   page_size                >= 1, any
 *   num_pages                pages of the caches >= 1
 *   max_pages                entries of a page_table row that may be read >= 1;
 *                            tokens past max_pages * page_size are not visible
 *   max_seq_len, max_kv_len  largest q_s and kv_len of the call.  Of a longer q_s the first max_seq_len
 *                            rows are computed.  With a longer kv_len, tokens from position max_kv_len on
 *                            are not visible; positions, and with them the causal order and the window,
 *                            stay those of kv_len, where the append put the tokens
 *   window                   0: none, else >= 1 tokens up to and including the query's
 *   sinks                    first tokens visible beside the window (>= 0)
 *   dtype                    q, k, v and out: RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   scale                    factor of the scores
 *   *_stride                 elements: pages, rows inside a page and heads of
 *                            both caches; rows of q, out, k_new, v_new; rows of page_table
 *   workspace_bytes          bytes at tables->workspace
 * One launch takes fewer than 2^24 workgroups: num_seqs * num_kv_heads * max_seq_len *
 * (num_q_heads / num_kv_heads) / 64 (its last two factors rounded up) is below that for the
 * attention, num_tokens * num_q_heads below 2^26 where a workspace is needed, and the bytes of
 * k_new below 2^36 for the append. */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t max_seq_len;
  int32_t max_kv_len;
  int32_t window;
  int32_t sinks;
  int32_t dtype;
  float scale;
  int64_t page_stride;
  int64_t row_stride;
  int64_t head_stride;
  int64_t q_token_stride;
  int64_t out_token_stride;
  int64_t new_token_stride;
  int64_t table_stride;
  int64_t workspace_bytes;
} rssm_paged_attention_desc;

/* Device tensors:
 *   k_cache, v_cache  [num_pages][page_size][num_kv_heads][head_dim] by the strides above (both alike)
 *   k_new, v_new      [num_tokens][num_kv_heads][head_dim] (append only)
 *   q, out            [num_tokens][num_q_heads][head_dim] (attention only)
 *   lse               [num_tokens][num_q_heads] fp32 or NULL: natural logarithm of the sum of exp(scale q.k_j)
 *   page_table        [num_seqs][max_pages] int32
 *   seq_start         [num_seqs + 1] int32 ascending; kv_len [num_seqs] int32
 *   workspace         device memory of workspace_bytes, or NULL when 0 is needed
 * Guards against faults: seq_start is clamped to [0, num_tokens], a negative kv_len
 * to 0, and pages outside [0, num_pages) are neither read nor
 * written; a new token whose position is negative is not appended.  Two sequences may share
 * pages as long as neither appends to them.  Alignment: caches, q, out,
 * k_new, v_new and workspace 16 bytes, their strides multiples of 16 bytes; the others 4 bytes. */
typedef struct {
  void *k_cache;
  void *v_cache;
  const void *k_new;
  const void *v_new;
  const void *q;
  void *out;
  float *lse;
  const int32_t *page_table;
  const int32_t *seq_start;
  const int32_t *kv_len;
  void *workspace;
} rssm_paged_attention_tables;

/* Copy the new tokens' keys and values into the cache at their positions. */
rssm_status rssm_paged_append(const rssm_paged_attention_desc *desc, const rssm_paged_attention_tables *tables,
                              void *hip_stream);

/* Workspace of rssm_paged_attention for these scalars, in bytes (0 when the
 * query tiles fill the device without splitting the token axis). */
rssm_status rssm_paged_attention_workspace(const rssm_paged_attention_desc *desc, int64_t *bytes);

/* Enqueue the attention on `hip_stream`.  Arithmetic: scores, maxima, sums and
 * outputs in fp32 on the matrix cores.  For their product with V, 16-bit dtypes round
 * the softmax weights once to the input dtype when max_seq_len * (num_q_heads /
 * num_kv_heads) > 16, and take them in two parts (16 bits and more) otherwise; fp16
 * weights below 2^-21 of the row's largest are within 2^-32 of it.  A value that a query may not
 * see never reaches its output, non-finite values included. */
rssm_status rssm_paged_attention(const rssm_paged_attention_desc *desc, const rssm_paged_attention_tables *tables,
                                 void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_PAGED_ATTENTION_H */

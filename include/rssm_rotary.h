/*
 * rssm_rotary.h -- C ABI of rotary positions in librssm_materialize (MI355X, gfx950): new queries
 * and keys of an attention layer are turned by their positions, and the keys and values appended to
 * the paged cache that rssm_paged_attention reads, in one pass.
 *
 * Sequence s's rows seq_start[s] .. seq_start[s+1] - 1 are its last tokens before kv_len[s], as in
 * rssm_paged_attention.h; token i of the rows is turned by its position p (positions[i] if given).  Of each
 * head the first rot_dim elements are turned in pairs i < rot_dim / 2, elements (2i, 2i + 1) when
 * interleaved, (i, i + rot_dim / 2) otherwise:
 *     (a, b) <- factor (a cos(p f_i) - b sin(p f_i), a sin(p f_i) + b cos(p f_i)),  f = inv_freq
 * and the rest of the head passes through.  Scaled variants for long contexts are frequencies and a factor.
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_ROTARY_H
#define RSSM_ROTARY_H

#include <stdint.h>

#include "rssm_materialize.h" /* dtype codes, rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side scalars.
 *   num_seqs, num_tokens     sequences; rows of q / k_new / v_new (>= 0)
 *   num_q_heads              heads of q, 0: no queries
 *   num_kv_heads             heads of k_new and v_new, 0: no keys and values (the cache fields are ignored)
 *   head_dim                 64 or 128
 *   rot_dim                  a multiple of 16 in [16, head_dim]
 *   interleaved              0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1)
 *   page_size, num_pages     as in rssm_paged_attention_desc
 *   max_pages                entries of a page_table row
 *   dtype                    q, q_out, k, v: RSSM_F32 | RSSM_BF16 | RSSM_F16
 *   factor                   of the sines and cosines (finite)
 *   *_stride                 elements: pages, rows inside a page and heads of both
 *                            caches; rows of q, q_out, k_new and v_new (one stride); rows of page_table
 * num_tokens is below 2^24 and each kind of heads in [0, 4096]. */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t rot_dim;
  int32_t interleaved;
  int32_t page_size;
  int32_t num_pages;
  int32_t max_pages;
  int32_t dtype;
  float factor;
  int64_t page_stride;
  int64_t row_stride;
  int64_t head_stride;
  int64_t q_token_stride;
  int64_t q_out_token_stride;
  int64_t k_token_stride;
  int64_t v_token_stride;
  int64_t table_stride;
} rssm_rotary_desc;

/* Device tensors:
 *   q, q_out          [num_tokens][num_q_heads][head_dim] (q_out may be q itself)
 *   k_new, v_new      [num_tokens][num_kv_heads][head_dim]
 *   k_cache, v_cache  [num_pages][page_size][num_kv_heads][head_dim] by the strides above (both alike)
 *   page_table        [num_seqs][max_pages] int32
 *   seq_start         [num_seqs + 1] int32 ascending; kv_len [num_seqs] int32
 *   positions         [num_tokens] int32 or NULL (the token's place in the cache).  It sets the angle only
 *   inv_freq          [rot_dim / 2] fp32, finite
 * Without keys and with positions, seq_start and kv_len may be NULL.  Rows of no sequence are left
 * untouched (without seq_start all rows are turned).  Guards against faults: as in rssm_paged_append; a token
 * that the append skips (negative position, page outside the pool) still has its query turned.  kv_len counts the new
 * tokens: rows that rssm_page_extend refused must have none here, or their new tokens overwrite their last ones.
 * Alignment: q, q_out, k_new, v_new and caches 16 bytes, their strides multiples of 16 bytes; the others 4 bytes. */
typedef struct {
  const void *q;
  void *q_out;
  const void *k_new;
  const void *v_new;
  void *k_cache;
  void *v_cache;
  const int32_t *page_table;
  const int32_t *seq_start;
  const int32_t *kv_len;
  const int32_t *positions;
  const float *inv_freq;
} rssm_rotary_tables;

/* Enqueue on `hip_stream`.  Angles are products and remainders in 64 bits (any int32 position), sines and
 * cosines and the rest fp32; each output is rounded once.  Values, and the elements of a head past rot_dim, are the
 * inputs' bytes. */
rssm_status rssm_rotary_append(const rssm_rotary_desc *desc, const rssm_rotary_tables *tables, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_ROTARY_H */

// rssm_rotary.hip -- host side of rssm_rotary.h: argument checks and the
// launch on the caller's stream.
#include "rssm_rotary.h"

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "rotary_kernel.h"
#include "rssm_host.h"

namespace {

using namespace rssm;

rssm_status check_stride(int64_t v, int64_t least, int64_t es, const char* n) {
  if (v < least) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is below the dense size", n);
  if (v > (int64_t(1) << 40)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s exceeds 2^40 elements", n);
  if ((v * es) % 16 != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s must be a multiple of 16 bytes", n);
  return RSSM_OK;
}

rssm_status check_desc(const rssm_rotary_desc* d) {
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->num_seqs < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", d->num_seqs);
  if (d->num_tokens < 0 || d->num_tokens >= (1 << 24))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_tokens must be in [0, 2^24) (got %d)", d->num_tokens);
  if (d->num_q_heads < 0 || d->num_q_heads > 4096)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_q_heads must be in [0, 4096] (got %d)", d->num_q_heads);
  if (d->num_kv_heads < 0 || d->num_kv_heads > 4096)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_kv_heads must be in [0, 4096] (got %d)", d->num_kv_heads);
  if (d->dtype < RSSM_F32 || d->dtype > RSSM_F8E4M3) return fail(RSSM_ERR_INVALID_ARGUMENT, "unknown dtype %d", d->dtype);
  if (d->dtype > RSSM_F16)
    return fail(RSSM_ERR_UNSUPPORTED, "dtype must be f32, bf16 or f16 (got %s)", dtype_name(d->dtype));
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(RSSM_ERR_UNSUPPORTED, "no compiled instance for head_dim=%d (64, 128)", d->head_dim);
  if (d->rot_dim < 16 || d->rot_dim > d->head_dim || d->rot_dim % 16 != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "rot_dim must be a multiple of 16 in [16, head_dim] (got %d)", d->rot_dim);
  if (d->interleaved != 0 && d->interleaved != 1)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "interleaved must be 0 or 1 (got %d)", d->interleaved);
  if (!std::isfinite(d->factor)) return fail(RSSM_ERR_INVALID_ARGUMENT, "factor must be finite");
  const int64_t es = d->dtype == RSSM_F32 ? 4 : 2, D = d->head_dim;
  rssm_status st = RSSM_OK;
  if (d->num_q_heads > 0) {
    st = check_stride(d->q_token_stride, d->num_q_heads * D, es, "q_token_stride");
    if (st == RSSM_OK) st = check_stride(d->q_out_token_stride, d->num_q_heads * D, es, "q_out_token_stride");
  }
  if (st == RSSM_OK && d->num_kv_heads > 0) {
    if (d->page_size < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "page_size must be >= 1 (got %d)", d->page_size);
    if (d->num_pages < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_pages must be >= 1 (got %d)", d->num_pages);
    if (d->max_pages < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "max_pages must be >= 1 (got %d)", d->max_pages);
    if (d->table_stride < d->max_pages || d->table_stride > (int64_t(1) << 40))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "table_stride must be in [max_pages, 2^40]");
    st = check_stride(d->page_stride, D, es, "page_stride");
    if (st == RSSM_OK) st = check_stride(d->row_stride, D, es, "row_stride");
    if (st == RSSM_OK) st = check_stride(d->head_stride, D, es, "head_stride");
    if (st == RSSM_OK) st = check_stride(d->k_token_stride, d->num_kv_heads * D, es, "k_token_stride");
    if (st == RSSM_OK) st = check_stride(d->v_token_stride, d->num_kv_heads * D, es, "v_token_stride");
  }
  return st;
}

struct Ptr { const void* p; const char* n; size_t align; };

template <int n>
rssm_status check_ptrs(const Ptr (&p)[n], bool optional) {
  for (const Ptr& e : p) {
    if (e.p == nullptr && !optional) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
    if (e.p != nullptr && !aligned(e.p, e.align))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  }
  return RSSM_OK;
}

template <int DT>
const void* of_dim(int head_dim) {
  return head_dim == 64 ? reinterpret_cast<const void*>(&rotary_kernel<DT, 64>)
                        : reinterpret_cast<const void*>(&rotary_kernel<DT, 128>);
}

}  // namespace

extern "C" rssm_status rssm_rotary_append(const rssm_rotary_desc* d, const rssm_rotary_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  const Ptr opt[] = {{t->q, "q", 16}, {t->q_out, "q_out", 16}, {t->k_new, "k_new", 16}, {t->v_new, "v_new", 16},
                     {t->k_cache, "k_cache", 16}, {t->v_cache, "v_cache", 16}, {t->page_table, "page_table", 4},
                     {t->seq_start, "seq_start", 4}, {t->kv_len, "kv_len", 4}, {t->positions, "positions", 4},
                     {t->inv_freq, "inv_freq", 4}};
  st = check_ptrs(opt, true);
  if (st != RSSM_OK) return st;
  if (d->num_tokens == 0 || (d->num_q_heads == 0 && d->num_kv_heads == 0)) return RSSM_OK;
  const Ptr freq[] = {{t->inv_freq, "inv_freq", 4}};
  st = check_ptrs(freq, false);
  if (st == RSSM_OK && d->num_q_heads > 0) {
    const Ptr need[] = {{t->q, "q", 16}, {t->q_out, "q_out", 16}};
    st = check_ptrs(need, false);
  }
  if (st == RSSM_OK && d->num_kv_heads > 0) {
    const Ptr need[] = {{t->k_new, "k_new", 16}, {t->v_new, "v_new", 16}, {t->k_cache, "k_cache", 16},
                        {t->v_cache, "v_cache", 16}, {t->page_table, "page_table", 4}};
    st = check_ptrs(need, false);
  }
  if (st == RSSM_OK && (d->num_kv_heads > 0 || t->positions == nullptr)) {
    const Ptr need[] = {{t->seq_start, "seq_start", 4}, {t->kv_len, "kv_len", 4}};
    st = check_ptrs(need, false);
  }
  if (st != RSSM_OK) return st;
  if (t->seq_start != nullptr && d->num_seqs == 0) return RSSM_OK;
  RotaryArgs a;
  a.q = static_cast<const char*>(t->q);
  a.q_out = static_cast<char*>(t->q_out);
  a.k_new = static_cast<const char*>(t->k_new);
  a.v_new = static_cast<const char*>(t->v_new);
  a.k = static_cast<char*>(t->k_cache);
  a.v = static_cast<char*>(t->v_cache);
  a.table = t->page_table;
  a.seq_start = t->seq_start;
  a.kv_len = t->kv_len;
  a.positions = t->positions;
  a.inv_freq = t->inv_freq;
  a.page_stride = d->page_stride;
  a.row_stride = d->row_stride;
  a.head_stride = d->head_stride;
  a.q_stride = d->q_token_stride;
  a.qo_stride = d->q_out_token_stride;
  a.k_stride = d->k_token_stride;
  a.v_stride = d->v_token_stride;
  a.table_stride = d->table_stride;
  a.num_seqs = d->num_seqs;
  a.num_tokens = d->num_tokens;
  a.Hq = d->num_q_heads;
  a.Hkv = d->num_kv_heads;
  a.rot_dim = d->rot_dim;
  a.interleaved = d->interleaved;
  a.page_size = d->page_size;
  a.num_pages = d->num_pages;
  a.max_pages = d->max_pages;
  a.factor = d->factor;
  const int passes = (d->num_q_heads + 2 * d->num_kv_heads + 64 / (d->head_dim / 16) - 1) / (64 / (d->head_dim / 16));
  a.shares = d->num_tokens < 4096 ? std::min(passes, 8) : 1;
  a.units = d->num_tokens * a.shares;
  if (verbose())
    std::fprintf(stderr, "[rssm_rotary_append] %s tokens=%d heads=%d/%d dim=%d of %d shares=%d\n", dtype_name(d->dtype),
                 d->num_tokens, d->num_q_heads, d->num_kv_heads, d->rot_dim, d->head_dim, a.shares);
  const void* fn = d->dtype == RSSM_F32 ? of_dim<kF32>(d->head_dim)
                   : d->dtype == RSSM_BF16 ? of_dim<kBF16>(d->head_dim) : of_dim<kF16>(d->head_dim);
  void* params[] = {&a};
  hipError_t e = hipLaunchKernel(fn, dim3((static_cast<unsigned>(a.units) + 3) / 4), dim3(kRotaryBlock), params, 0,
                                 static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of rotary_append failed: %s", hipGetErrorString(e));
  return RSSM_OK;
}

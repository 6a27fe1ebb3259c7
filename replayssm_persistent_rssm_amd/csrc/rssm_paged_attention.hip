// rssm_paged_attention.hip -- host side of rssm_paged_attention.h: argument
// checks, the split of the key axis, launches on the caller's stream.
#include "rssm_paged_attention.h"

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "paged_inst.h"
#include "rssm_host.h"

namespace rssm {
const void* paged_f32_for(int which, int head_dim);
const void* paged_bf16_for(int which, int head_dim);
const void* paged_f16_for(int which, int head_dim);
}  // namespace rssm

namespace {

using namespace rssm;

const void* kernel_for(int which, const rssm_paged_attention_desc* d) {
  switch (d->dtype) {
    case RSSM_F32: return paged_f32_for(which, d->head_dim);
    case RSSM_BF16: return paged_bf16_for(which, d->head_dim);
    default: return paged_f16_for(which, d->head_dim);
  }
}

int elem_bytes(int dt) { return dt == RSSM_F32 ? 4 : 2; }

rssm_status check_stride(int64_t v, int64_t least, int64_t es, const char* n) {
  if (v < least) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is below the dense size", n);
  if (v > (int64_t(1) << 40)) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s exceeds 2^40 elements", n);
  if ((v * es) % 16 != 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s must be a multiple of 16 bytes", n);
  return RSSM_OK;
}

rssm_status check_desc(const rssm_paged_attention_desc* d, bool append) {
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->num_seqs < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_seqs must be >= 0 (got %d)", d->num_seqs);
  if (d->num_tokens < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_tokens must be >= 0 (got %d)", d->num_tokens);
  if (d->num_kv_heads < 1 || d->num_kv_heads > 65536)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_kv_heads must be in [1, 65536] (got %d)", d->num_kv_heads);
  if (d->page_size < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "page_size must be >= 1 (got %d)", d->page_size);
  if (d->num_pages < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "num_pages must be >= 1 (got %d)", d->num_pages);
  if (d->max_pages < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "max_pages must be >= 1 (got %d)", d->max_pages);
  if (d->dtype < RSSM_F32 || d->dtype > RSSM_F8E4M3) return fail(RSSM_ERR_INVALID_ARGUMENT, "unknown dtype %d", d->dtype);
  if (d->dtype > RSSM_F16)
    return fail(RSSM_ERR_UNSUPPORTED, "dtype must be f32, bf16 or f16 (got %s)", dtype_name(d->dtype));
  if (d->head_dim != 64 && d->head_dim != 128)
    return fail(RSSM_ERR_UNSUPPORTED, "no compiled instance for head_dim=%d (64, 128)", d->head_dim);
  const int64_t es = elem_bytes(d->dtype), D = d->head_dim;
  rssm_status st = check_stride(d->page_stride, D, es, "page_stride");
  if (st == RSSM_OK) st = check_stride(d->row_stride, D, es, "row_stride");
  if (st == RSSM_OK) st = check_stride(d->head_stride, D, es, "head_stride");
  if (st != RSSM_OK) return st;
  if (d->table_stride < d->max_pages || d->table_stride > (int64_t(1) << 40))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "table_stride must be in [max_pages, 2^40]");
  if (append) return check_stride(d->new_token_stride, d->num_kv_heads * D, es, "new_token_stride");
  if (d->num_q_heads < 1 || d->num_q_heads > 65536 || d->num_q_heads % d->num_kv_heads != 0)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_kv_heads (%d) must divide num_q_heads (%d, in [1, 65536])",
                d->num_kv_heads, d->num_q_heads);
  if (d->max_seq_len < 0 || d->max_seq_len > (1 << 24))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "max_seq_len must be in [0, 2^24] (got %d)", d->max_seq_len);
  if (static_cast<int64_t>(d->max_seq_len) * (d->num_q_heads / d->num_kv_heads) > (1 << 30))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "max_seq_len*(num_q_heads/num_kv_heads) exceeds 2^30");
  if (d->max_kv_len < 0 || d->max_kv_len > (1 << 30))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "max_kv_len must be in [0, 2^30] (got %d)", d->max_kv_len);
  if (d->window < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "window must be >= 0 (got %d)", d->window);
  if (d->sinks < 0 || d->sinks > (1 << 30))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "sinks must be in [0, 2^30] (got %d)", d->sinks);
  if (!(d->scale > 0.0f) || !std::isfinite(d->scale))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "scale must be positive and finite");
  st = check_stride(d->q_token_stride, d->num_q_heads * D, es, "q_token_stride");
  if (st == RSSM_OK) st = check_stride(d->out_token_stride, d->num_q_heads * D, es, "out_token_stride");
  if (st != RSSM_OK) return st;
  if (d->workspace_bytes < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace_bytes must be >= 0");
  return RSSM_OK;
}

struct Ptr { const void* p; const char* n; size_t align; };

rssm_status check_ptrs(const Ptr* p, int n, bool optional) {
  for (int i = 0; i < n; ++i) {
    if (p[i].p == nullptr && !optional) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", p[i].n);
    if (p[i].p != nullptr && !aligned(p[i].p, p[i].align))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", p[i].n, p[i].align);
  }
  return RSSM_OK;
}

struct Plan {
  bool rows16;        // at most 16 rows a (sequence, key/value head): the streaming kernel
  int row_tiles, nsplit, split_tiles;
};

// The split of the key axis.  Row tiles: none when they give every compute unit a
// workgroup, otherwise as many as fit two each in one round (2,000 new tokens over 40,000, 4 query heads
// and one key/value head of 128: 210 us with 504 workgroups, 299 with 567), of at least 2 tiles of keys (3 times 5
// new tokens over 4,000, 16 / 4 heads of 64: 17.6 us, 20.6 with 4).  Single tokens: up to 4,096
// workgroups, because ragged lengths leave many of them without work (64 requests of
// 1 to 8,192 tokens, 32 / 8 heads of 128: 229 us with 1,024, 210 with 2,048, 212 with 4,096, 224 with
// 8,192), each of at least 8 tiles (short caches) to 32 (long ones, where joining costs more: one
// request of 131,071 tokens 60.5 us with 32, 65.3 with 16).
Plan plan_of(const rssm_paged_attention_desc* d) {
  Plan p;
  const int64_t group = d->num_q_heads / d->num_kv_heads;
  const int64_t rows = d->max_seq_len * group;
  p.rows16 = rows <= 16;
  const int64_t T = p.rows16 ? 32 : 64, tile_rows = p.rows16 ? 16 : 64 * paged_row_blocks(d->dtype);
  p.row_tiles = static_cast<int>(std::max<int64_t>(1, (rows + tile_rows - 1) / tile_rows));
  int64_t tiles = (d->max_kv_len + T - 1) / T;
  if (d->window > 0) {
    const int64_t span = tile_rows / group + 2;   // positions of a row tile
    tiles = std::min(tiles, (d->sinks + T - 1) / T + (d->window + span) / T + 2);
  }
  const int64_t items = static_cast<int64_t>(d->num_seqs) * d->num_kv_heads * p.row_tiles;
  const int64_t kFill = p.rows16 ? 4096 : 512;
  const int64_t kLeast = p.rows16 ? std::min<int64_t>(32, std::max<int64_t>(8, tiles / 32)) : 2;
  p.nsplit = 1;
  p.split_tiles = 1 << 30;
  if (items > 0 && items <= (p.rows16 ? kFill : kFill / 2) && tiles >= 2 * kLeast) {
    const int64_t want = p.rows16 ? (kFill + items - 1) / items : kFill / items;
    const int64_t per = std::max(kLeast, (tiles + want - 1) / want);
    const int64_t n = (tiles + per - 1) / per;
    if (n > 1) {
      p.nsplit = static_cast<int>(n);
      p.split_tiles = static_cast<int>(per);
    }
  }
  return p;
}

int64_t workspace_of(const rssm_paged_attention_desc* d, const Plan& p) {
  if (p.nsplit == 1) return 0;
  return static_cast<int64_t>(d->num_tokens) * d->num_q_heads * p.nsplit * (d->head_dim + 2) * 4;
}

void fill_args(PagedArgs* a, const rssm_paged_attention_desc* d, const rssm_paged_attention_tables* t) {
  a->k = static_cast<char*>(t->k_cache);
  a->v = static_cast<char*>(t->v_cache);
  a->k_new = static_cast<const char*>(t->k_new);
  a->v_new = static_cast<const char*>(t->v_new);
  a->q = static_cast<const char*>(t->q);
  a->out = static_cast<char*>(t->out);
  a->lse = t->lse;
  a->table = t->page_table;
  a->seq_start = t->seq_start;
  a->kv_len = t->kv_len;
  a->part_o = nullptr;
  a->part_ml = nullptr;
  a->page_stride = d->page_stride;
  a->row_stride = d->row_stride;
  a->head_stride = d->head_stride;
  a->q_stride = d->q_token_stride;
  a->out_stride = d->out_token_stride;
  a->new_stride = d->new_token_stride;
  a->table_stride = d->table_stride;
  // exact division of j < 2^31: with 2^(l-1) < size <= 2^l, ceil(2^(31+l) / size) fits 32 bits
  int l = 0;
  while ((int64_t(1) << l) < d->page_size) ++l;
  a->page_shift = 31 + l;
  a->page_magic = static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d->page_size - 1) / d->page_size);
  a->num_seqs = d->num_seqs;
  a->num_tokens = d->num_tokens;
  a->Hq = d->num_q_heads;
  a->Hkv = d->num_kv_heads;
  a->group = 1;
  a->page_size = d->page_size;
  a->num_pages = d->num_pages;
  a->max_pages = d->max_pages;
  a->max_seq_len = d->max_seq_len;
  a->max_kv_len = d->max_kv_len;
  a->window = std::min(d->window, 1 << 30);   // no cache is longer
  a->sinks = d->sinks;
  a->scale_log2 = d->scale * 1.4426950408889634f;
  a->row_tiles = 1;
  a->nsplit = 1;
  a->split_tiles = 1 << 30;
}

rssm_status check_grid(int64_t grid, const char* name) {
  if (grid > kMaxWorkgroups)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "%s needs %lld workgroups, more than one launch takes (2^24 - 1)", name,
                static_cast<long long>(grid));
  return RSSM_OK;
}

rssm_status launch(const void* fn, int64_t grid, void** params, void* stream, const char* name) {
  hipError_t e = hipLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(kPagedBlock), params, 0,
                                 static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of %s failed: %s", name, hipGetErrorString(e));
  return RSSM_OK;
}

}  // namespace

extern "C" {

rssm_status rssm_paged_append(const rssm_paged_attention_desc* d, const rssm_paged_attention_tables* t,
                              void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, true);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0 || d->num_tokens == 0) return RSSM_OK;
  const Ptr need[] = {{t->k_cache, "k_cache", 16}, {t->v_cache, "v_cache", 16}, {t->k_new, "k_new", 16},
                      {t->v_new, "v_new", 16}, {t->page_table, "page_table", 4}, {t->seq_start, "seq_start", 4},
                      {t->kv_len, "kv_len", 4}};
  st = check_ptrs(need, 7, false);
  if (st != RSSM_OK) return st;
  PagedArgs a;
  fill_args(&a, d, t);
  int head_vecs = d->head_dim * elem_bytes(d->dtype) / 16;
  const int64_t work = static_cast<int64_t>(d->num_tokens) * d->num_kv_heads * head_vecs;
  void* params[] = {&a, &head_vecs};
  const void* fn = d->dtype == RSSM_F32 ? reinterpret_cast<const void*>(&paged_append_kernel<4>)
                                        : reinterpret_cast<const void*>(&paged_append_kernel<2>);
  const int64_t grid = (work + kPagedBlock - 1) / kPagedBlock;
  st = check_grid(grid, "paged_append");
  if (st != RSSM_OK) return st;
  return launch(fn, grid, params, hip_stream, "paged_append");
}

rssm_status rssm_paged_attention_workspace(const rssm_paged_attention_desc* d, int64_t* bytes) {
  clear_error();
  rssm_status st = check_desc(d, false);
  if (st != RSSM_OK) return st;
  if (bytes == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = workspace_of(d, plan_of(d));
  return RSSM_OK;
}

rssm_status rssm_paged_attention(const rssm_paged_attention_desc* d, const rssm_paged_attention_tables* t,
                                 void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, false);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_seqs == 0 || d->num_tokens == 0 || d->max_seq_len == 0) return RSSM_OK;
  const Ptr need[] = {{t->k_cache, "k_cache", 16}, {t->v_cache, "v_cache", 16}, {t->q, "q", 16}, {t->out, "out", 16},
                      {t->page_table, "page_table", 4}, {t->seq_start, "seq_start", 4}, {t->kv_len, "kv_len", 4}};
  st = check_ptrs(need, 7, false);
  if (st != RSSM_OK) return st;
  const Ptr opt[] = {{t->lse, "lse", 4}, {t->workspace, "workspace", 16}};
  st = check_ptrs(opt, 2, true);
  if (st != RSSM_OK) return st;
  const Plan p = plan_of(d);
  const int64_t need_bytes = workspace_of(d, p);
  if (need_bytes > 0 && (t->workspace == nullptr || d->workspace_bytes < need_bytes))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace of %lld bytes is needed (got %lld)",
                static_cast<long long>(need_bytes),
                static_cast<long long>(t->workspace == nullptr ? 0 : d->workspace_bytes));
  PagedArgs a;
  fill_args(&a, d, t);
  a.group = d->num_q_heads / d->num_kv_heads;
  a.row_tiles = p.row_tiles;
  a.nsplit = p.nsplit;
  a.split_tiles = p.split_tiles;
  const int64_t out_rows = static_cast<int64_t>(d->num_tokens) * d->num_q_heads;
  if (p.nsplit > 1) {
    a.part_o = static_cast<float*>(t->workspace);
    a.part_ml = a.part_o + out_rows * p.nsplit * d->head_dim;
  }
  if (verbose())
    std::fprintf(stderr, "[rssm_paged_attention] %s seqs=%d heads=%d/%d dim=%d %s row_tiles=%d splits=%d\n",
                 dtype_name(d->dtype), d->num_seqs, d->num_q_heads, d->num_kv_heads, d->head_dim,
                 p.rows16 ? "rows" : "tiles", p.row_tiles, p.nsplit);
  void* params[] = {&a};
  const int64_t grid = static_cast<int64_t>(d->num_seqs) * d->num_kv_heads * p.row_tiles * p.nsplit;
  // few rows with many splits: a workgroup a row (one request of 131,071 tokens, 32 / 4 heads of 128: 55.0 us,
  // 63.6 with a wavefront a row; 40 new tokens over 20,000, 16 / 4 heads: 35.5, 38.7).  Otherwise a wavefront
  // a row: no difference at 8 splits (64 requests up to 8,192: 212.2, 212.5) or with thousands of rows
  // (255 new tokens, 16 heads: 71.8 and 72.0)
  const bool share = p.nsplit > 16 && out_rows < 4096;
  const int64_t join_grid = share ? out_rows : (out_rows + 3) / 4;
  st = check_grid(grid, "paged_attention");
  if (st == RSSM_OK && p.nsplit > 1) st = check_grid(join_grid, "paged_join");
  if (st != RSSM_OK) return st;
  st = launch(kernel_for(p.rows16 ? kPagedRow : kPagedTile, d), grid, params, hip_stream, "paged_attention");
  if (st != RSSM_OK || p.nsplit == 1) return st;
  return launch(kernel_for(share ? kPagedJoinShare : kPagedJoin, d), join_grid, params, hip_stream, "paged_join");
}

}  // extern "C"

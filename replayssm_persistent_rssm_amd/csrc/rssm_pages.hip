// rssm_pages.hip -- host side of rssm_pages.h: argument checks and launches on
// the caller's stream.
#include "rssm_pages.h"

#include <algorithm>
#include <cstdio>

#include "pages_kernel.h"
#include "rssm_host.h"

namespace {

using namespace rssm;

enum : int { kExtend, kFork, kRelease, kCompact, kCopy };

constexpr int64_t kPagesGrid = 4096;   // workgroups that take the tasks of a copying kernel in turn

rssm_status check_desc(const rssm_pages_desc* d, int op) {
  if (d == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (op != kCompact && (d->num_items < 0 || d->num_items > (1 << 20)))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_items must be in [0, 2^20] (got %d)", d->num_items);
  if (d->num_pages < 1 || d->num_pages > (1 << 30))
    return fail(RSSM_ERR_INVALID_ARGUMENT, "num_pages must be in [1, 2^30] (got %d)", d->num_pages);
  if (op != kCopy) {
    if (d->num_rows < 1 || d->num_rows > (1 << 20))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "num_rows must be in [1, 2^20] (got %d)", d->num_rows);
    if (d->max_pages < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "max_pages must be >= 1 (got %d)", d->max_pages);
    if (d->page_size < 1) return fail(RSSM_ERR_INVALID_ARGUMENT, "page_size must be >= 1 (got %d)", d->page_size);
    if (d->table_stride < d->max_pages || d->table_stride > (int64_t(1) << 40))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "table_stride must be in [max_pages, 2^40]");
  }
  if (op == kFork || op == kCompact || op == kCopy) {
    if (d->num_caches < 0 || d->num_caches > 65535)
      return fail(RSSM_ERR_INVALID_ARGUMENT, "num_caches must be in [0, 65535] (got %d)", d->num_caches);
    if (d->page_bytes < 16 || d->page_bytes % 16 != 0 || d->page_bytes > (int64_t(1) << 30))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "page_bytes must be a multiple of 16 in [16, 2^30]");
    if (d->page_stride < d->page_bytes || d->page_stride % 16 != 0 || d->page_stride > (int64_t(1) << 46) / d->num_pages)
      return fail(RSSM_ERR_INVALID_ARGUMENT, "page_stride must be a multiple of 16 of at least page_bytes, num_pages*page_stride at most 2^46");
    if (op == kFork && d->token_bytes != 0 &&
        (d->token_bytes < 16 || d->token_bytes % 16 != 0 || d->token_bytes > d->page_bytes ||
         d->token_bytes * d->page_size != d->page_bytes))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "token_bytes must be 0 or a multiple of 16 that page_size times gives page_bytes");
  }
  if (d->workspace_bytes < 0) return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace_bytes must be >= 0");
  return RSSM_OK;
}

// Bytes: claim [rows], first, plan and fresh [items], list and moved [pages], count.
int64_t workspace_of(const rssm_pages_desc* d) {
  return 4 * (static_cast<int64_t>(d->num_rows) + 3 * static_cast<int64_t>(d->num_items) + 2 * static_cast<int64_t>(d->num_pages) + 4);
}

struct Ptr { const void* p; const char* n; size_t align; };

template <int n>
rssm_status check_ptrs(const Ptr (&p)[n], bool optional = false) {
  for (const Ptr& e : p) {
    if (e.p == nullptr && !optional) return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is NULL", e.n);
    if (e.p != nullptr && !aligned(e.p, e.align))
      return fail(RSSM_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", e.n, e.align);
  }
  return RSSM_OK;
}

rssm_status check_rows(const rssm_pages_tables* t) {
  const Ptr need[] = {{t->page_table, "page_table", 4}, {t->kv_len, "kv_len", 4}, {t->page_ref, "page_ref", 4}};
  return check_ptrs(need);
}

rssm_status check_workspace(const rssm_pages_desc* d, const rssm_pages_tables* t) {
  const Ptr ws[] = {{t->workspace, "workspace", 16}};
  rssm_status st = check_ptrs(ws, true);
  if (st != RSSM_OK) return st;
  const int64_t need = workspace_of(d);
  if (t->workspace == nullptr || d->workspace_bytes < need)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "workspace of %lld bytes is needed (got %lld)", static_cast<long long>(need),
                static_cast<long long>(t->workspace == nullptr ? 0 : d->workspace_bytes));
  return RSSM_OK;
}

rssm_status check_caches(const rssm_pages_desc* d, const rssm_pages_tables* t) {
  if (d->num_caches == 0) return RSSM_OK;
  const Ptr need[] = {{t->cache_ptrs, "cache_ptrs", 8}};
  return check_ptrs(need);
}

void fill_args(PagesArgs* a, const rssm_pages_desc* d, const rssm_pages_tables* t) {
  a->cache_ptrs = t->cache_ptrs;
  a->table = t->page_table;
  a->kv_len = t->kv_len;
  a->ref = t->page_ref;
  a->src = t->src;
  a->dst = t->dst;
  a->lengths = t->lengths;
  a->status = t->status;
  a->live = t->live;
  int32_t* w = static_cast<int32_t*>(t->workspace);
  a->claim = w;
  a->first = w == nullptr ? nullptr : w + d->num_rows;
  a->plan = w == nullptr ? nullptr : a->first + d->num_items;
  a->fresh = w == nullptr ? nullptr : a->plan + d->num_items;
  a->list = w == nullptr ? nullptr : a->fresh + d->num_items;
  a->moved = w == nullptr ? nullptr : a->list + d->num_pages;
  a->count = w == nullptr ? nullptr : a->moved + d->num_pages;
  a->table_stride = d->table_stride;
  a->page_bytes = d->page_bytes;
  a->page_stride = d->page_stride;
  a->token_bytes = d->token_bytes;
  a->num_items = d->num_items;
  a->num_rows = d->num_rows;
  a->max_pages = d->max_pages;
  a->num_pages = d->num_pages;
  a->page_size = d->page_size;
  a->num_caches = d->num_caches;
  a->chunks = static_cast<int32_t>((d->page_bytes + kPagesChunk - 1) / kPagesChunk);
}

rssm_status launch(const void* fn, int64_t grid, int block, PagesArgs* a, void* stream, const char* name) {
  void* params[] = {a};
  hipError_t e = hipLaunchKernel(fn, dim3(static_cast<unsigned>(grid)), dim3(block), params, 0, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(RSSM_ERR_HIP, "launch of %s failed: %s", name, hipGetErrorString(e));
  return RSSM_OK;
}

template <bool FORK>
rssm_status launch_plan(PagesArgs* a, void* stream, const char* name) {
  if (a->num_items > kPlanFew) return launch(reinterpret_cast<const void*>(&pages_plan_kernel<FORK>), 1, kPlanBlock, a, stream, name);
  if (a->num_pages > 256 * kPlanPages)
    return launch(reinterpret_cast<const void*>(&pages_plan_few_kernel<FORK, 1024>), 1, 1024, a, stream, name);
  return launch(reinterpret_cast<const void*>(&pages_plan_few_kernel<FORK, 256>), 1, 256, a, stream, name);
}

// The tasks of a copying kernel are counted in 32 bits; 2^31 of them would be 32 TiB.
rssm_status check_tasks(int64_t items, int64_t per, int64_t more, const char* name) {
  if (items > 0 && per > ((int64_t(1) << 31) - more) / items)
    return fail(RSSM_ERR_INVALID_ARGUMENT, "%s has more than 2^31 pieces of %d bytes to look at", name, kPagesChunk);
  return RSSM_OK;
}

void say(const char* name, const rssm_pages_desc* d) {
  if (verbose())
    std::fprintf(stderr, "[rssm_%s] items=%d rows=%d pages=%d caches=%d\n", name, d->num_items, d->num_rows, d->num_pages,
                 d->num_caches);
}

}  // namespace

extern "C" {

rssm_status rssm_pages_workspace(const rssm_pages_desc* d, int64_t* bytes) {
  clear_error();
  rssm_status st = check_desc(d, kExtend);
  if (st != RSSM_OK) return st;
  if (bytes == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "bytes is NULL");
  *bytes = workspace_of(d);
  return RSSM_OK;
}

rssm_status rssm_page_extend(const rssm_pages_desc* d, const rssm_pages_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, kExtend);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_items == 0) return RSSM_OK;
  st = check_rows(t);
  if (st != RSSM_OK) return st;
  const Ptr need[] = {{t->dst, "dst", 4}, {t->lengths, "lengths", 4}, {t->status, "status", 4}};
  st = check_ptrs(need);
  if (st == RSSM_OK) st = check_workspace(d, t);
  if (st != RSSM_OK) return st;
  PagesArgs a;
  fill_args(&a, d, t);
  say("page_extend", d);
  return launch_plan<false>(&a, hip_stream, "page_extend");
}

rssm_status rssm_page_fork(const rssm_pages_desc* d, const rssm_pages_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, kFork);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_items == 0) return RSSM_OK;
  st = check_rows(t);
  if (st != RSSM_OK) return st;
  const Ptr need[] = {{t->src, "src", 4}, {t->dst, "dst", 4}, {t->status, "status", 4}}, opt[] = {{t->lengths, "lengths", 4}};
  st = check_ptrs(need);
  if (st == RSSM_OK) st = check_ptrs(opt, true);
  if (st == RSSM_OK) st = check_caches(d, t);
  if (st == RSSM_OK) st = check_workspace(d, t);
  if (st != RSSM_OK) return st;
  PagesArgs a;
  fill_args(&a, d, t);
  st = check_tasks(d->num_items, 1 + static_cast<int64_t>(d->num_caches) * a.chunks, 0, "page_fork");
  if (st != RSSM_OK) return st;
  say("page_fork", d);
  st = launch_plan<true>(&a, hip_stream, "page_fork (plan)");
  if (st != RSSM_OK) return st;
  const int64_t tasks = d->num_items * (1 + static_cast<int64_t>(d->num_caches) * a.chunks);
  return launch(reinterpret_cast<const void*>(&pages_fork_kernel), std::min(tasks, kPagesGrid), kPagesBlock, &a, hip_stream, "page_fork");
}

rssm_status rssm_page_release(const rssm_pages_desc* d, const rssm_pages_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, kRelease);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_items == 0) return RSSM_OK;
  st = check_rows(t);
  if (st != RSSM_OK) return st;
  const Ptr need[] = {{t->dst, "dst", 4}}, opt[] = {{t->lengths, "lengths", 4}};
  st = check_ptrs(need);
  if (st == RSSM_OK) st = check_ptrs(opt, true);
  if (st != RSSM_OK) return st;
  PagesArgs a;
  fill_args(&a, d, t);
  say("page_release", d);
  return launch(reinterpret_cast<const void*>(&pages_release_kernel), d->num_items, kPagesBlock, &a, hip_stream, "page_release");
}

rssm_status rssm_page_compact(const rssm_pages_desc* d, const rssm_pages_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, kCompact);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  st = check_rows(t);
  if (st != RSSM_OK) return st;
  const Ptr need[] = {{t->live, "live", 4}};
  rssm_pages_desc e = *d;
  e.num_items = 0;                       // not read by this call
  st = check_ptrs(need);
  if (st == RSSM_OK) st = check_caches(&e, t);
  if (st == RSSM_OK) st = check_workspace(&e, t);
  if (st != RSSM_OK) return st;
  PagesArgs a;
  fill_args(&a, &e, t);
  st = check_tasks(d->num_pages / 2, static_cast<int64_t>(d->num_caches) * a.chunks, d->num_rows, "page_compact");
  if (st != RSSM_OK) return st;
  say("page_compact", &e);
  st = launch(reinterpret_cast<const void*>(&pages_pack_kernel), 1, kPlanBlock, &a, hip_stream, "page_compact (plan)");
  if (st != RSSM_OK) return st;
  // at most half of the pages move; how many do is known on the device alone
  const int64_t tasks = d->num_rows + static_cast<int64_t>(d->num_pages / 2) * d->num_caches * a.chunks;
  return launch(reinterpret_cast<const void*>(&pages_move_kernel), std::min(tasks, kPagesGrid), kPagesBlock, &a, hip_stream, "page_compact");
}

rssm_status rssm_page_copy(const rssm_pages_desc* d, const rssm_pages_tables* t, void* hip_stream) {
  clear_error();
  rssm_status st = check_desc(d, kCopy);
  if (st != RSSM_OK) return st;
  if (t == nullptr) return fail(RSSM_ERR_INVALID_ARGUMENT, "tables is NULL");
  if (d->num_items == 0 || d->num_caches == 0) return RSSM_OK;
  const Ptr need[] = {{t->src, "src", 4}, {t->dst, "dst", 4}};
  st = check_ptrs(need);
  if (st == RSSM_OK) st = check_caches(d, t);
  if (st != RSSM_OK) return st;
  PagesArgs a;
  fill_args(&a, d, t);
  st = check_tasks(d->num_items, static_cast<int64_t>(d->num_caches) * a.chunks, 0, "page_copy");
  if (st != RSSM_OK) return st;
  say("page_copy", d);
  const int64_t tasks = static_cast<int64_t>(d->num_items) * d->num_caches * a.chunks;
  return launch(reinterpret_cast<const void*>(&pages_copy_kernel), std::min(tasks, kPagesGrid), kPagesBlock, &a, hip_stream, "page_copy");
}

}  // extern "C"

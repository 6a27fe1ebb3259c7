/*
 * rssm_pages.h -- C ABI of the pages of a paged cache in librssm_materialize (MI355X, gfx950): extending,
 * forking, releasing, compacting and copying.  The counterpart, for attention layers, of what the
 * materialize operation does for state pools: a prefix of a request becomes a request of its own.
 *
 * The pool is described by three tables that live on the device:
 *   page_table [num_rows][max_pages]  pages of each request's row in order, -1 where none
 *   kv_len     [num_rows]             tokens of each row, which holds ceil(kv_len / page_size) pages
 *   page_ref   [num_pages]            rows that hold each page; 0: the page is free
 * They are all that is kept: a page is taken by its index, the lowest free one first, items of a call in
 * their order, so that results do not depend on timing.  One table serves any number of caches (keys and
 * values of every layer): page p of cache i is the page_bytes bytes at cache_ptrs[i] + p * page_stride.
 *
 * Plain C types only.  Every pointer is DEVICE memory owned by the caller;
 * the library allocates nothing and never synchronises.
 */
#ifndef RSSM_PAGES_H
#define RSSM_PAGES_H

#include <stdint.h>

#include "rssm_materialize.h" /* rssm_status, rssm_last_error */

#ifdef __cplusplus
extern "C" {
#endif

#define RSSM_PAGE_OK 0       /* done */
#define RSSM_PAGE_NONE 1     /* too few free pages: the row is as it was */
#define RSSM_PAGE_REFUSED 2  /* a row outside the table, named twice, of negative or too great length, or (fork)
                                a destination that holds tokens: the row is as it was */
#define RSSM_PAGE_SHARED 3   /* (extend) the row's last page is not full and counted more than once (another row
                                holds it too): fork the row first; the row is as it was */

/* Host-side scalars (each entry point reads those it names).
 *   num_items      rows or pages that the call works on >= 0, at most 2^20
 *   num_rows       rows of the table >= 1, at most 2^20
 *   max_pages      entries of a row >= 1
 *   num_pages      pages of the pool >= 1, at most 2^30
 *   page_size      tokens of a page >= 1
 *   num_caches     entries of cache_ptrs >= 0, at most 65535
 *   table_stride   elements between rows of page_table >= max_pages
 *   page_bytes     bytes of a page in each cache, a multiple of 16
 *   page_stride    bytes between pages, a multiple of 16, >= page_bytes
 *   token_bytes    a multiple of 16 that page_size times gives page_bytes, when a page holds its tokens
 *                  one after another (a fork then copies the filled ones alone); 0: laid out otherwise
 *   workspace_bytes  bytes at tables->workspace
 * Items (compact: half of the pages) times caches times the 16 KiB pieces of a page are below 2^31. */
typedef struct {
  int32_t num_items;
  int32_t num_rows;
  int32_t max_pages;
  int32_t num_pages;
  int32_t page_size;
  int32_t num_caches;
  int64_t table_stride;
  int64_t page_bytes;
  int64_t page_stride;
  int64_t token_bytes;
  int64_t workspace_bytes;
} rssm_pages_desc;

/* Device tensors:
 *   cache_ptrs   [num_caches] addresses (16-byte aligned) of the caches (copy, fork, compact)
 *   page_table, kv_len, page_ref as above
 *   src, dst     [num_items] int32: rows (fork), pages (copy); dst alone: rows (extend, release)
 *   lengths      [num_items] int32: tokens to add (extend), tokens of the fork (fork; NULL: all of the
 *                source's), tokens that stay (release; NULL: none)
 *   status       [num_items] int32, written (extend, fork): RSSM_PAGE_OK, _NONE, _REFUSED or _SHARED.  A row whose
 *                extend is not RSSM_PAGE_OK has its old kv_len: its new tokens must not be appended (their places, counted
 *                back from kv_len, are those of its last tokens, on pages that other rows may hold too)
 *   live         [1] int32, written (compact): pages in use, which are the pages 0 .. live - 1 afterwards
 *   workspace    device memory of workspace_bytes (extend, fork, compact)
 * Contract: calls on one pool are ordered (one stream, or events); the tables agree with one another (a pool starts with page_table -1, kv_len 0 and page_ref 0
 * and is changed by these calls alone, apart from page counts that the caller takes or gives back for
 * itself).  As a guard against faults, pages outside the pool are neither read nor written.
 * Alignment: workspace 16 bytes, cache_ptrs 8, the others 4. */
typedef struct {
  const int64_t *cache_ptrs;
  int32_t *page_table;
  int32_t *kv_len;
  int32_t *page_ref;
  const int32_t *src;
  const int32_t *dst;
  const int32_t *lengths;
  int32_t *status;
  int32_t *live;
  void *workspace;
} rssm_pages_tables;

/* Workspace of extend, fork and compact for these scalars, in bytes (the largest of the three). */
rssm_status rssm_pages_workspace(const rssm_pages_desc *desc, int64_t *bytes);

/* Rows dst[i] grow by lengths[i] tokens: the pages they lack are taken, kv_len is advanced.  An item gets its
 * pages when they and those of all items before it are free, otherwise none (RSSM_PAGE_NONE); items that need no
 * page always succeed. */
rssm_status rssm_page_extend(const rssm_pages_desc *desc, const rssm_pages_tables *tables, void *hip_stream);

/* Rows dst[i], which are empty, become the first min(lengths[i], kv_len[src[i]]) tokens of rows src[i]: full pages are
 * shared (counted once more), the tokens of a last page that is not full are copied to a page of the fork's
 * own, in every cache.  Several items may have one source; sources are
 * taken as they were when the call began.  Of rows named twice as a destination the first item counts.  These calls
 * never write to a shared page again: rows grow on pages of their own. */
rssm_status rssm_page_fork(const rssm_pages_desc *desc, const rssm_pages_tables *tables, void *hip_stream);

/* Rows dst[i] keep their first lengths[i] tokens (none without lengths); pages past them are given back, those that
 * no other row holds become free.  Rows outside the table are skipped; a length at or above the row's, or a
 * negative one, changes nothing.  A row may be named twice. */
rssm_status rssm_page_release(const rssm_pages_desc *desc, const rssm_pages_tables *tables, void *hip_stream);

/* The pages in use move to the front of the pool: the i-th page in use at or past their number moves to the i-th free page
 * before it, in every cache; page_table and page_ref follow.  Pages that the caller counts for itself move as well. */
rssm_status rssm_page_compact(const rssm_pages_desc *desc, const rssm_pages_tables *tables, void *hip_stream);

/* Page dst[i] becomes a copy of page src[i] in every cache (num_items pairs; no page among dst twice or
 * among src too).  The tables are neither read nor written. */
rssm_status rssm_page_copy(const rssm_pages_desc *desc, const rssm_pages_tables *tables, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* RSSM_PAGES_H */

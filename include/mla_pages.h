/*
 * Paged MLA for GB300 (sm_103a): pages of the cache handed out, shared, copied
 * and freed on the device.  C ABI.
 *
 * A pool of num_pages pages has a reference count for each: how many table
 * rows name it.  A page with count 0 is free.  Table rows hold page ids, -1
 * where a request has no page.
 *
 *   mla_page_resize  every request gets the pages that its new length needs and
 *                    gives back those behind (length 0: all of them);
 *   mla_page_fork    requests continue as several (a beam step, samples of one
 *                    prompt): full pages are shared, a started page is copied.
 *
 * Pages are handed out in ascending id, the lowest free one first, to the
 * missing entries in the order of the rows and, within a row, of the columns.
 * So the results depend on the inputs only.
 *
 * Conventions as in mla_decode.h: caller-owned device buffers, asynchronous on
 * `stream`, no allocation, no synchronisation, an mla_status return, device
 * errors OR-ed into word 0 of the workspace (read it with mla_query_status).
 * The calls can be captured into a CUDA graph.  Calls on one pool's counts
 * follow each other on a stream (or are ordered by the caller).
 */
#ifndef MLA_PAGES_H_
#define MLA_PAGES_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MLA_DEV_NO_PAGES = 512, /* the pool ran out: entries that got no page are -1 */
  MLA_DEV_BAD_REFS = 1024 /* a page was given back more often than its count, or had a count below 0; its count is 0
                             before pages are handed out */
};

typedef struct {
  int32_t batch;             /* B >= 1 requests */
  int32_t num_pages;         /* pool size, >= 1, at most 2^30 */
  int32_t max_pages_per_req; /* columns of both tables, >= 1; * 64 and * B must fit in int32 */
  int32_t table_stride;      /* int32 elements between rows of page_table (>= max_pages_per_req) */
  int32_t out_stride;        /* of page_table_out */
} mla_page_resize_dims;

/* Bytes of workspace; 0 on invalid dimensions. */
size_t mla_page_resize_workspace_size(int32_t batch, int32_t max_pages_per_req, int32_t num_pages);

/*
 * Request b is to hold ceil(new_lens[b] / 64) pages in its first columns.  An
 * entry >= 0 among them stays; an entry below 0 receives a free page (count 1);
 * an entry >= 0 behind them is given back (count - 1, a free page at 0) and
 * becomes -1.  All pages are given back before any is handed out.
 *
 *   new_lens    int32 [B]; in [0, max_pages_per_req * 64] (else
 *               MLA_DEV_BAD_SEQ_LEN; clamped)
 *   page_table  int32 [B][table_stride].  An id >= num_pages raises
 *               MLA_DEV_BAD_PAGE_ID; it stays where it is needed, and counts nothing
 *   page_refs   int32 [num_pages]
 *   page_table_out, page_refs_out: int32; each may be its input itself (with the
 *               same stride), and must not overlap it otherwise
 *   workspace   256-byte aligned
 * Outputs and workspace overlap nothing else (MLA_ERR_INVALID_ARG; a table is
 * its rows' columns, what lies between them is free).
 * One kernel.
 */
int mla_page_resize(const mla_page_resize_dims* d, const int32_t* new_lens, const int32_t* page_table,
                    const int32_t* page_refs, int32_t* page_table_out, int32_t* page_refs_out, void* workspace,
                    size_t workspace_bytes, void* stream);

typedef struct {
  int32_t sources;           /* rows of page_table and seq_lens, >= 1 */
  int32_t children;          /* rows of page_table_out, >= 1 */
  int32_t num_layers;        /* caches that share the page table, >= 1, at most 65535 */
  int32_t num_pages;         /* pool size, >= 1; num_pages * 64 must fit in int32 */
  int32_t max_pages_per_req; /* columns of both tables, >= 1; * 64 and * children must fit in int32 */
  int32_t table_stride;      /* int32 elements between rows of page_table (>= max_pages_per_req) */
  int32_t out_stride;        /* of page_table_out */
  int32_t kv_dtype;          /* mla_kv_dtype of the caches */
  int64_t layer_stride;      /* bytes from one layer's cache to the next, a multiple of 16 and at least a cache
                                (ignored for one layer) */
} mla_page_fork_dims;

/* Bytes of workspace; 0 on invalid dimensions. */
size_t mla_page_fork_workspace_size(int32_t sources, int32_t children, int32_t max_pages_per_req, int32_t num_pages);

/*
 * Child c continues source s = src[c] of L = seq_lens[s] tokens: its row shares
 * the source's L / 64 full pages (count + 1 each); where L % 64 tokens remain
 * it receives a free page (count 1) into which their rows are copied, in every
 * layer; the entries behind are -1.  The source keeps what it has (give it back
 * with mla_page_resize when it ends).
 *
 *   src         int32 [children]; -1: an empty row.  Another value outside
 *               [0, sources): MLA_DEV_BAD_INDEX and an empty row
 *   seq_lens    int32 [sources]; in [0, max_pages_per_req * 64] (else
 *               MLA_DEV_BAD_SEQ_LEN; clamped)
 *   page_table  int32 [sources][table_stride].  A needed id outside
 *               [0, num_pages): MLA_DEV_BAD_PAGE_ID and -1 in its place
 *   page_refs, page_refs_out: int32 [num_pages]; may be the same
 *   kv_cache    num_layers caches [num_pages][64][576], 16-byte aligned
 *   page_table_out: int32 [children][out_stride]; the two tables must not
 *               overlap, counted from their first to their last element
 *   workspace   256-byte aligned
 * Outputs and workspace overlap nothing else (as for mla_page_resize; no buffer
 * lies in the caches, which is not looked at).
 * Two kernels.
 */
int mla_page_fork(const mla_page_fork_dims* d, const int32_t* src, const int32_t* seq_lens, const int32_t* page_table,
                  const int32_t* page_refs, void* kv_cache, int32_t* page_table_out, int32_t* page_refs_out,
                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PAGES_H_ */

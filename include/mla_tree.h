/*
 * Paged MLA for GB300 (sm_103a): trees of drafted tokens over the paged latent
 * cache.  C ABI.
 *
 * A speculative step gives every request a few drafted tokens that form a
 * tree: several continuations are tried at once, and the attention of all of
 * them is one call.  Request b's n_b = cu_q_lens[b + 1] - cu_q_lens[b] nodes
 * are the last n_b of its seq_lens[b] cached tokens (their rows are in the
 * cache already, see mla_rope.h and mla_kv_pack.h), node i in slot
 * seq_lens[b] - n_b + i.  A node's parent comes before it (parents[] holds its
 * index within the request, -1: none; several nodes may have none).
 *
 *   mla_decode_tree   attention of the nodes: node i sees the tokens before the
 *                     tree, its ancestors and itself;
 *   mla_tree_commit   after the verification (see mla_verify.h): the rows of
 *                     the accepted nodes move together, in every layer's cache.
 *
 * A chain (parents[i] = i - 1) gives mla_prefill's results without a window,
 * bit for bit.
 *
 * Conventions as in mla_decode.h: caller-owned device buffers, asynchronous
 * on `stream`, no allocation, no synchronisation, an mla_status return.  The
 * calls can be captured into a CUDA graph and read lengths, offsets, parents
 * and tables anew at every replay.  Results depend on the inputs and the
 * dimensions only, bit for bit.
 */
#ifndef MLA_TREE_H_
#define MLA_TREE_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"
#include "mla_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MLA_TREE_MAX_NODES = 256 /* of a request */ };

enum { MLA_DEV_BAD_TREE = 128 /* a parent that is not -1 .. i - 1 (the node then has none), or a request with more than
                                 MLA_TREE_MAX_NODES nodes (left out; its outputs are not written) */ };

/* Bytes of workspace mla_decode_tree needs for these dimensions on `device`:
 * mla_prefill's and 32 bytes per node, whatever the lengths.  0 on invalid
 * dimensions or if the device cannot be queried. */
size_t mla_decode_tree_workspace_size(const mla_prefill_dims* d, int device);

/*
 * Attention of trees of drafted tokens: mla_prefill's dimensions, arguments,
 * layouts and limits (see mla_prefill.h, total_q nodes in all), without a
 * window, and
 *
 *   cu_q_lens   as for mla_prefill, with at most MLA_TREE_MAX_NODES nodes a
 *               request.  (Where offsets decrease, which is flagged, a token that two
 *               requests name gets either's outputs, seeing either's ancestors)
 *   parents     int32 [total_q]: each node's parent within its request, < its
 *               own index, or -1.  Entries from cu_q_lens[B] on are not read
 *
 * Every row below seq_lens[b] holds finite values, those of nodes that a node
 * does not see too.  out and lse as mla_prefill's; three kernels.  Device
 * errors are OR-ed into the status word of the workspace (mla_query_status).
 */
int mla_decode_tree(const mla_prefill_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                    const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_q_lens,
                    const int32_t* parents, float scale, float kv_scale, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream);

typedef struct {
  int32_t batch;             /* B >= 1 requests, at most 65535 (else MLA_ERR_UNSUPPORTED) */
  int32_t num_layers;        /* caches that share the page table, >= 1, at most 65535 */
  int32_t path_cols;         /* row length of path, >= 1 */
  int32_t num_pages;         /* pool size of each cache; valid page ids are [0, num_pages) */
  int32_t max_pages_per_req; /* columns of the page table a request may use; * 64 must fit in int32 */
  int32_t page_table_stride; /* int32 elements between page-table rows (>= max_pages_per_req) */
  int32_t kv_dtype;          /* mla_kv_dtype of the caches */
  int32_t reserved;          /* 0 */
  int64_t layer_stride;      /* bytes from one layer's cache to the next, a multiple of 16 and at least a cache
                                (ignored for one layer) */
} mla_tree_commit_dims;

/*
 * Keeps a request's accepted nodes: with base = seq_lens[b] - n_b and
 * a = num_path[b], the row of node path[b][k] moves to slot base + k for
 * k = 0 .. a - 1, in every layer, and new_lens[b] = base + a.  The rows behind
 * stay as they are, unused.
 *
 *   kv_cache    num_layers caches [num_pages][64][576], 16-byte aligned; only
 *               rows that receive another node's are written, so the pages from
 *               slot base on belong to the request alone
 *   page_table  int32 [B][page_table_stride]; read for the slots from base on
 *   seq_lens    int32 [B]; in [n_b, max_pages_per_req * 64]
 *   cu_q_lens   int32 [B + 1], non-decreasing from >= 0
 *   path        int32 [B][path_cols]: nodes, ascending, in [0, n_b)
 *   num_path    int32 [B]; in [0, min(n_b, path_cols)]; 0 drops all nodes
 *   new_lens    int32 [B]; like status, must not overlap the inputs, which every
 *               block reads (MLA_ERR_INVALID_ARG; of a table's row what is behind
 *               max_pages_per_req is free.  The cache is not looked at)
 *   status      int32 [1]; OR-ed in: MLA_DEV_BAD_SEQ_LEN, MLA_DEV_BAD_QUERY_RANGE,
 *               MLA_DEV_BAD_TREE (more than MLA_TREE_MAX_NODES nodes),
 *               MLA_DEV_BAD_INDEX (path or num_path): the request is left out
 *               and new_lens[b] = seq_lens[b]; MLA_DEV_BAD_PAGE_ID: a move that
 *               meets a bad page id is skipped.  The caller clears it
 * One kernel.
 */
int mla_tree_commit(const mla_tree_commit_dims* d, void* kv_cache, const int32_t* page_table, const int32_t* seq_lens,
                    const int32_t* cu_q_lens, const int32_t* path, const int32_t* num_path, int32_t* new_lens,
                    int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_TREE_H_ */

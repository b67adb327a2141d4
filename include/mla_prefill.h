/*
 * Paged MLA for GB300 (sm_103a): attention of chunks of new tokens over the
 * paged latent cache (prompt processing, chunked or mixed steps).  C ABI.
 *
 * The operation is the one of mla_decode.h (absorbed queries, one latent row
 * [c_kv (512) | k_pe (64)] per cached token, 64-token pages through a page
 * table) for requests that bring any number of new tokens each.  Request b's
 * n_b = cu_q_lens[b + 1] - cu_q_lens[b] new tokens are the last n_b of its
 * seq_lens[b] cached tokens (their rows are in the cache already, see
 * mla_kv_pack.h).  Its token i, at position p = seq_lens[b] - n_b + i, sees
 *
 *     window == 0:  the keys t <= p;
 *     window >= 1:  the keys t <= p with t > p - window (a sliding window of
 *                   `window` tokens, the token itself among them) or
 *                   t < num_sinks (a few first tokens that stay visible);
 *
 *     s_t = (q_nope . c_kv[t] + q_pe . k_pe[t]) * scale
 *     out = sum_t softmax(s)_t * c_kv[t],   lse = ln sum_t exp(s_t)
 *
 * The weights are rounded before they multiply the rows: to bf16 with a bf16
 * cache; with an e4m3 cache to f16, as shares of a reference that is at most the
 * row's greatest weight.  There a weight below 2^-25 (e^-17) of the greatest
 * counts as none, so that out misses at most 2^-25 of the greatest weight times
 * the sum of |c_kv[t]| over such keys.  (It shows where a few tokens take nearly
 * all the weight and have values near 0.)  lse counts every key in full.
 *
 * Key t is the row in slot t of the request.  On a cache that mla_evict (see
 * mla_evict.h) has shortened, slots are no longer positions: call without a
 * window there.
 *
 * Conventions as in mla_decode.h: caller-owned device buffers, asynchronous
 * on `stream`, no allocation, no synchronisation, an mla_status return, and
 * device errors OR-ed into the status word of the workspace (read it with
 * mla_query_status).  Three kernels per call.  The calls can be captured into
 * a CUDA graph; a captured call reads lengths, offsets and the page table anew
 * at every replay.  Results depend on the inputs and the dimensions only,
 * bit for bit.
 */
#ifndef MLA_PREFILL_H_
#define MLA_PREFILL_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MLA_DEV_BAD_QUERY_RANGE = 64 /* cu_q_lens does not start at 0, decreases or passes total_q; the request was
                                       left out and its rows of out and lse were not written */ };

typedef struct {
  int32_t batch;             /* B >= 1 requests */
  int32_t num_heads;         /* H >= 1 absorbed query heads */
  int32_t total_q;           /* rows of the query tensors in tokens, >= 1; total_q * H must fit in int32 */
  int32_t page_size;         /* must be 64 */
  int32_t num_pages;         /* pool size; valid page ids are [0, num_pages) */
  int32_t max_pages_per_req; /* columns of the page table a request may use; max_pages_per_req * 64 must fit in int32,
                                and so must the pages that all blocks of queries could visit,
                                (total_q * H / 128 + B) * max_pages_per_req; the blocks alone at most 2^30 (else
                                MLA_ERR_UNSUPPORTED) */
  int32_t page_table_stride; /* int32 elements between page-table rows (>= max_pages_per_req) */
  int32_t kv_dtype;          /* mla_kv_dtype */
} mla_prefill_dims;

/* Bytes of workspace mla_prefill needs for these dimensions on `device`: the
 * schedule and fp32 split partials, about 40 MB plus 36 bytes per 128 query
 * rows, whatever the lengths.  0 on invalid dimensions or if the device
 * cannot be queried. */
size_t mla_prefill_workspace_size(const mla_prefill_dims* d, int device);

/*
 *   q_nope      bf16 [total_q][H][512], contiguous, 32-byte aligned
 *   q_pe        bf16 [total_q][H][64],  contiguous, 32-byte aligned
 *   kv_cache    bf16 or e4m3 [num_pages][64][576], 16-byte aligned; an e4m3
 *               value means code * kv_scale.  A slot that no query of its
 *               request may see because it lies behind seq_lens[b] may hold
 *               anything; the others of a visited page hold finite values
 *   page_table  int32 [B][page_table_stride]; read only for the pages that a
 *               query sees (with a window: the sinks' and the windows' pages)
 *   seq_lens    int32 [B]; in [n_b, max_pages_per_req * 64] where n_b > 0
 *               (else MLA_DEV_BAD_SEQ_LEN; the length is clamped and tokens
 *               at negative positions see nothing: out = 0, lse = -inf)
 *   cu_q_lens   int32 [B + 1]: cu_q_lens[0] = 0, non-decreasing, at most
 *               total_q; n_b = 0 is a request without queries in this call.
 *               Rows of q, out and lse from cu_q_lens[B] on are not touched
 *   window      0: none; >= 1 (MLA_ERR_INVALID_ARG below 0)
 *   num_sinks   >= 0; without a window it changes nothing
 *   scale       softmax scale, > 0 and finite
 *   kv_scale    e4m3 cache: > 0 and finite; bf16 cache: ignored.
 *               scale * kv_scale * log2(e) must be finite and above 0 in fp32
 *   out         bf16 [total_q][H][512], 32-byte aligned
 *   lse         fp32 [total_q][H]
 *   workspace   >= mla_prefill_workspace_size bytes, 256-byte aligned; not
 *               shared by calls that may run concurrently
 */
int mla_prefill(const mla_prefill_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_q_lens, int32_t window,
                int32_t num_sinks, float scale, float kv_scale, void* out, float* lse, void* workspace,
                size_t workspace_bytes, void* stream);

/* Bytes of workspace mla_decode_window needs; d as for mla_decode, but
 * num_heads * q_len is not limited to 256 (B * q_len * H must fit in int32).
 * 0 on invalid dimensions. */
size_t mla_decode_window_workspace_size(const mla_dims* d, int device);

/*
 * Decode over a sliding window and a few first tokens: mla_decode's arguments
 * and layouts, with q_len = d->q_len tokens per request, each seeing the
 * window of `window` >= 1 tokens that ends with itself and the first
 * num_sinks >= 0 tokens.  Only the pages that hold them are read, so the
 * caller may have freed the others (their table entries are not looked at).
 * Not for a request that mla_evict has shortened, and its log-sum-exps are not
 * for mla_attn_mass (see mla_evict.h for both).
 * Works like mla_prefill with n_b = q_len for every request.
 */
int mla_decode_window(const mla_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                      const int32_t* page_table, const int32_t* seq_lens, int32_t window, int32_t num_sinks,
                      float scale, float kv_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_PREFILL_H_ */

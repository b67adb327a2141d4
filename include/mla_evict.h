/*
 * Paged MLA for GB300 (sm_103a): a cache kept within a budget by accumulated
 * attention weight.  C ABI.
 *
 * Two operations beside the decode of mla_decode.h and the chunks of
 * mla_prefill.h:
 *
 *   mla_attn_mass  adds up the softmax weight that a step's queries gave to
 *                  every cached token, over all heads and query positions;
 *   mla_evict      keeps, of every request that outgrew its budget, the
 *                  tokens of the greatest accumulated weight (and its first
 *                  and latest ones), and moves the rows kept behind the budget
 *                  into the places of the dropped ones.
 *
 * A step writes its rows (mla_kv_pack), attends (mla_decode, or mla_prefill
 * without a window), accumulates (mla_attn_mass, from the same queries and the
 * log-sum-exps that the attention returned) and, when a request is over its
 * budget, evicts.  What does not go together:
 *
 *   - A windowed or top-k step (mla_decode_window, mla_prefill with a window,
 *     mla_decode_sparse) and mla_attn_mass.  The mass is over every token up to
 *     the query's own; with a log-sum-exp over fewer keys exp(s - lse) is no
 *     share of a softmax (it may pass 1), and the pages of tokens outside a
 *     window, which the caller may have freed, would be read.
 *   - mla_evict and windows.  After an eviction a slot is no longer a position:
 *     the kept tokens from behind the budget, the latest among them, sit in
 *     whatever slots were free.  mla_decode_window and mla_prefill with a
 *     window choose keys by slot, so from then on the request is attended to
 *     without a window.
 *
 * mla_attn_mass takes the same number of queries for every request.  After a
 * ragged mla_prefill the caller gathers the last q_len tokens' queries and
 * log-sum-exps of each request, with q_len at most the fewest that one brought.
 *
 * Conventions as in mla_decode.h: caller-owned device
 * buffers, asynchronous on `stream`, no allocation, no synchronisation, an
 * mla_status return, device errors OR-ed into word 0 of the workspace (read
 * it with mla_query_status).  The calls can be captured into a CUDA graph.
 * Results depend on the inputs only, bit for bit.
 */
#ifndef MLA_EVICT_H_
#define MLA_EVICT_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace mla_attn_mass needs (the status words); 0 on invalid
 * dimensions.  d as for mla_decode, but num_heads * q_len is not limited. */
size_t mla_attn_mass_workspace_size(const mla_dims* d, int device);

/*
 * For request b with L = seq_lens[b] cached tokens and its q_len queries at
 * the positions L - q_len .. L - 1 (each sees the tokens up to its own):
 *
 *     mass_out[b][t] = (t < L - num_fresh ? mass[b][t] : 0)
 *                      + sum over positions i and heads h that see t of
 *                        exp(s_t - lse[b][i][h]),
 *     s_t = (q_nope . c_kv[t] + q_pe . k_pe[t]) * scale,     0 <= t < L.
 *
 * Entries t >= L are not touched.  A query row with lse = -inf (it saw
 * nothing) adds nothing.
 *
 *   d, q_nope, q_pe, kv_cache, page_table, seq_lens, scale, kv_scale: as for
 *               mla_decode, and scale * kv_scale * log2(e) finite and above 0
 *               in fp32; every page of a request's L tokens is read
 *   lse         fp32 [B][q_len][H], as the attention over all tokens up to the
 *               query's own returned it
 *   num_fresh   the last num_fresh tokens start from zero instead of mass
 *               (a step's new tokens), >= 0
 *   mass        fp32 [B][mass_cols], or null: every token starts from zero
 *   mass_cols   row length of mass and mass_out, >= 1; seq_lens[b] is in
 *               [q_len, min(mass_cols, max_pages_per_req * 64)] (else
 *               MLA_DEV_BAD_SEQ_LEN, and the length is clamped)
 *   mass_out    fp32 [B][mass_cols]; may be mass itself
 *   workspace   >= mla_attn_mass_workspace_size bytes, 256-byte aligned
 * Returns MLA_ERR_UNSUPPORTED where B * max_pages_per_req * 64 is beyond 2^30
 * or B * q_len * H does not fit in int32.
 */
int mla_attn_mass(const mla_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                  const int32_t* page_table, const int32_t* seq_lens, const float* lse, int32_t num_fresh, float scale,
                  float kv_scale, const float* mass, float* mass_out, int32_t mass_cols, void* workspace,
                  size_t workspace_bytes, void* stream);

typedef struct {
  int32_t batch;             /* B >= 1 requests */
  int32_t mass_cols;         /* row length of mass, positions and their outputs, >= 1; mass_cols or budget beyond 2^30
                                or batch beyond 65535: MLA_ERR_UNSUPPORTED */
  int32_t num_pages;         /* pool size; valid page ids are [0, num_pages) */
  int32_t max_pages_per_req; /* columns of the page table a request may use */
  int32_t page_table_stride; /* int32 elements between page-table rows (>= max_pages_per_req) */
  int32_t kv_dtype;          /* mla_kv_dtype of the cache */
  int32_t budget;            /* tokens a request keeps at most, >= 1 */
  int32_t num_sinks;         /* first tokens that always stay, >= 0 */
  int32_t num_recent;        /* latest tokens that always stay, >= 0; num_sinks + num_recent <= budget */
} mla_evict_dims;

/* Bytes of workspace mla_evict needs: the lists of moves, 8 bytes per request
 * and token of its budget.  0 for batch < 1 or budget < 1. */
size_t mla_evict_workspace_size(int32_t batch, int32_t budget);

/*
 * Request b has L = seq_lens[b] cached tokens, token t with the accumulated
 * weight mass[b][t] and the position positions[b][t] in the whole
 * conversation (t itself where positions is null).  With k = min(L, budget)
 * it keeps the k first tokens in this order: the firm ones, which are those
 * of a position below num_sinks or among the num_recent positions that end
 * with the request's greatest; then the others by weight, the greater first
 * (a NaN last); the lower slot t first among equals.  Kept tokens in the
 * slots below k stay where they are; the j-th free slot below k, ascending,
 * receives the j-th kept token from the slots from k on, ascending, with its
 * cache row.  Then, for slots t < k, with o the old slot of the token that is
 * now in slot t:
 *
 *     new_lens[b] = k, kept[b][t] = o, mass_out[b][t] = mass[b][o],
 *     positions_out[b][t] = positions[b][o];   kept[b][t] = -1 for t >= k.
 *
 * Entries of mass_out and positions_out from k on are not touched.  The rows
 * behind k stay in the cache, unused.  (Attention without a window does not
 * depend on the order of the kept rows; the tokens of later steps follow in
 * slot k.)
 *
 *   mass        fp32 [B][mass_cols]; seq_lens[b] is in
 *               [0, min(mass_cols, max_pages_per_req * 64)] (else
 *               MLA_DEV_BAD_SEQ_LEN, and the length is clamped)
 *   positions   int32 [B][mass_cols], >= 0, or null (positions_out is then
 *               not written and may be null).  Null is right for a request's
 *               first eviction only: after it a slot is no longer a position
 *   kv_cache    [num_pages][64][576], 16-byte aligned; only rows that receive
 *               a token are written, so a page may be shared with another
 *               request only while all of its slots stay where they are in
 *               both (for instance pages of sink tokens).  A move with a bad
 *               page id is skipped and raises MLA_DEV_BAD_PAGE_ID
 *   new_lens    int32 [B]; may be seq_lens itself
 *   kept        int32 [B][budget]
 *   mass_out, positions_out: [B][mass_cols]; may be mass and positions
 *   workspace   >= mla_evict_workspace_size bytes, 256-byte aligned
 */
int mla_evict(const mla_evict_dims* d, const float* mass, const int32_t* positions, const int32_t* seq_lens,
              const int32_t* page_table, void* kv_cache, int32_t* new_lens, int32_t* kept, float* mass_out,
              int32_t* positions_out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_EVICT_H_ */

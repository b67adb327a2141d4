/*
 * Paged MLA for GB300 (sm_103a): rotary positions of a step's query and key
 * parts, with the cache write of its rows.  C ABI.
 *
 * mla_decode and its relatives take q_pe and cached k_pe that are rotated
 * already.  mla_rope_pack rotates both and writes the step's rows into the
 * paged cache, in one launch, for any number of new tokens per request: what
 * mla_kv_pack (see mla_kv_pack.h) does for the same number of rows each, with
 * the rotation before it.
 *
 * With the first R = rotary_dim of the 64 dimensions rotated, pair i < R / 2
 * turns by theta_i = position * f_i radians:
 *
 *     out_a = amplitude * (a cos theta_i - b sin theta_i)
 *     out_b = amplitude * (a sin theta_i + b cos theta_i)
 *
 *     interleaved:  a, b = x[2 i], x[2 i + 1]
 *     halves:       a, b = x[i], x[i + R / 2]
 *
 * The dimensions from R on pass unchanged.  A frequency is kept as a 64-bit
 * fraction of a turn, so that position * f_i modulo a turn is an integer
 * product and its error does not grow with the position beyond that of f_i in
 * 64-bit floating point (2^-52 relative).
 */
#ifndef MLA_ROPE_H_
#define MLA_ROPE_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"
#include "mla_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Filled by mla_rope_plan_init; read on the host during each call. */
typedef struct {
  uint64_t turn[32];   /* f_i / (2 pi) in units of 2^-64 */
  int32_t rotary_dim;  /* R: 16, 32, 48 or 64 */
  int32_t interleaved; /* 1: pairs (2 i, 2 i + 1); 0: halves */
  float amplitude;
  int32_t reserved;
} mla_rope_plan;

/*
 * Frequencies in radians a position, out[i] for i < R / 2, R = rotary_dim:
 * f_i = base^(-2 i / R), and for contexts `factor` times longer than trained
 * for
 *
 *     original_len == 0:  f_i / factor
 *     original_len > 0:   g_i f_i + (1 - g_i) f_i / factor, g_i in [0, 1]:
 *                         pairs that turn often in original_len positions
 *                         stay, the slow ones stretch.
 *
 * The two functions differ in g between the pairs that turn `fast` and `slow`
 * times, which are whole other frequencies (R = 64, base 10000, factor 40,
 * original_len 4096, fast 32, slow 1: pairs 11 to 22, pair 20 by a factor of
 * 4.3).  Take the one that the weights were trained with:
 *
 *   mla_rope_frequencies           linear in the turns, as the method was
 *       published: g_i = (r_i - slow) / (fast - slow), limited to [0, 1], with
 *       r_i = original_len f_i / (2 pi) turns;
 *   mla_rope_frequencies_by_index  linear in the pair's index, between whole
 *       indices: what DeepSeek-V3's configuration means by these parameters
 *       (factor, original_len, fast and slow = beta_fast and beta_slow).
 *       g_i = 1 - (i - lo) / (hi - lo), limited to [0, 1], with
 *       lo = max(floor(I(fast)), 0), hi = min(ceil(I(slow)), R - 1) and
 *       I(n) = R ln(original_len / (2 pi n)) / (2 ln base), the index that turns
 *       n times.  Where hi <= lo, pairs up to lo stay and the others stretch.
 *
 * Host only.  MLA_ERR_INVALID_ARG for a null pointer, base < 1, factor < 1,
 * original_len < 0 or fast <= slow (looked at where original_len > 0; by
 * index, there, also for base == 1 or slow <= 0), or values that are not
 * finite; MLA_ERR_UNSUPPORTED for another rotary_dim.
 */
int mla_rope_frequencies(int32_t rotary_dim, double base, double factor, int32_t original_len, double fast,
                         double slow, double* out);
int mla_rope_frequencies_by_index(int32_t rotary_dim, double base, double factor, int32_t original_len, double fast,
                                  double slow, double* out);

/* A plan of any frequencies, each in [0, 2 pi) (else MLA_ERR_INVALID_ARG, as
 * for an amplitude that is not finite and above 0).  Host only. */
int mla_rope_plan_init(int32_t rotary_dim, int32_t interleaved, float amplitude, const double* frequencies,
                       mla_rope_plan* plan);

typedef struct {
  int32_t batch;             /* B >= 1 requests */
  int32_t num_heads;         /* H >= 1 query heads, at most 65536 (else MLA_ERR_UNSUPPORTED) */
  int32_t total_q;           /* tokens in all, >= 1; total_q * H must fit in int32 */
  int32_t num_pages;         /* pool size; valid page ids are [0, num_pages) */
  int32_t max_pages_per_req; /* columns of the page table a request may use; * 64 must fit in int32 */
  int32_t page_table_stride; /* int32 elements between page-table rows (>= max_pages_per_req) */
  int32_t kv_dtype;          /* mla_kv_dtype of the cache */
  int32_t reserved;          /* 0 */
  int64_t q_token_stride;    /* bf16 elements between tokens and between heads of q_pe: multiples of 8, */
  int64_t q_head_stride;     /* >= 64 (one head or one token: ignored) */
  int64_t row_stride;        /* bf16 elements between rows: a multiple of 8, >= 576 (one token: ignored) */
} mla_rope_dims;

/*
 * Request b's n_b = cu_q_lens[b + 1] - cu_q_lens[b] new tokens are the last
 * n_b of its seq_lens[b] cached ones; its token i goes to slot
 * seq_lens[b] - n_b + i.
 *
 *   plan        see above (host memory)
 *   q_pe        bf16 [total_q][H][64] with the strides of d, 16-byte aligned
 *   rows        bf16 [total_q][576] with row_stride, 16-byte aligned: c_kv, then
 *               k_pe before its rotation
 *   positions   int32 [total_q], or null: the token's slot.  (Nodes of a tree
 *               have the position of their depth; see mla_tree.h)
 *   page_table  int32 [B][page_table_stride]; read for the new tokens' slots
 *   seq_lens    int32 [B]; in [n_b, max_pages_per_req * 64] where n_b > 0 (else
 *               MLA_DEV_BAD_SEQ_LEN and the request is left out: neither its
 *               queries nor its rows are written)
 *   cu_q_lens   int32 [B + 1] as for mla_prefill (else MLA_DEV_BAD_QUERY_RANGE and
 *               the request is left out; a token that two others name where the
 *               offsets decrease is the last one's, and the first's slot keeps
 *               its row); tokens from cu_q_lens[B] on are not touched
 *   kv_scale    e4m3 cache: a normal, finite number with a finite reciprocal;
 *               bf16 cache: ignored
 *   q_out       bf16 [total_q][H][64], contiguous, 16-byte aligned: the rotated
 *               queries, rounded once.  May be q_pe itself where that is
 *               contiguous; must not overlap it otherwise
 *   kv_cache    [num_pages][64][576], 16-byte aligned; only the new rows are
 *               written.  c_kv as mla_kv_pack writes it; the rotated k_pe is
 *               rounded once, to bf16 or to the e4m3 code nearest to
 *               value / kv_scale (saturated to +-448).  A row with a bad page id
 *               is not written (MLA_DEV_BAD_PAGE_ID)
 *   status      int32 [1] (device), OR-ed into; the caller clears it
 *
 * q_out and status overlap neither one another nor rows, positions, page_table,
 * seq_lens and cu_q_lens (MLA_ERR_INVALID_ARG; what lies between the rows of a
 * strided buffer is free).  Rows of the cache that the call writes are not
 * among its inputs (which is not looked at).
 *
 * One kernel, asynchronous on `stream`; it can be captured into a CUDA graph.
 */
int mla_rope_pack(const mla_rope_dims* d, const mla_rope_plan* plan, const void* q_pe, const void* rows,
                  const int32_t* positions, const int32_t* page_table, const int32_t* seq_lens,
                  const int32_t* cu_q_lens, float kv_scale, void* q_out, void* kv_cache, int32_t* status,
                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_ROPE_H_ */

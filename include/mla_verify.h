/*
 * Paged MLA for GB300 (sm_103a): verification of drafted tokens against the
 * target's probabilities, from given random numbers.  C ABI.
 *
 * A request's nodes form a tree (see mla_tree.h): node 0 is the last token
 * that is decided already, the others are drafts below it, and row i of the
 * target's probabilities is the distribution of the token that follows node i.
 * From node 0 the call walks down the accepted drafts, in such a way that the
 * tokens it returns are distributed as the target's own:
 *
 *     at node c:  w = p[c], z = 1; for c's children j, ascending, with token x:
 *       draft given (children drawn independently from q[c]):
 *         accepted if accept[j] * z * q[c][x] < w[x];
 *         else w = max(w - z q[c], 0), z = sum w;
 *       no draft (fixed proposals, e.g. a drafter's best few):
 *         accepted if accept[j] * z < w[x];
 *         else z = max(z - w[x], 0), w[x] = 0;
 *     on the first accepted child the walk goes on there; where none is, the
 *     last token is the lowest y with sum_{y' <= y} w[y'] > sample[b] * sum w.
 *
 * (Where w has become all zeros, by rounding, the last token comes from p[c].)
 * Fixed proposals take one pass over a row whatever is rejected.  Sampled drafts
 * take a further one for each rejected sibling, dearer each time (65536 tokens:
 * 2 us for the first, 10 for the second, 28 in all for 3, 1.3 ms for 40).
 * Sums run in integers, units of 2^-60, so that they are exact whatever their
 * order (an entry below 2^-36 is rounded to them).  The product of a test is
 * compared exactly, but for drafts after a rejection, where it is formed in
 * 64-bit floating point.
 *
 * Conventions as in mla_decode.h: caller-owned device buffers, asynchronous on
 * `stream`, no allocation, no synchronisation, an mla_status return.  One
 * kernel; it can be captured into a CUDA graph.  Results depend on the inputs
 * only.
 */
#ifndef MLA_VERIFY_H_
#define MLA_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#include "mla_decode.h"
#include "mla_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MLA_DEV_BAD_PROBS = 256 /* a row to sample from has no positive entry; the last token is -1 */ };

typedef struct {
  int32_t batch;          /* B >= 1 requests, at most 2^27 */
  int32_t total_q;        /* nodes in all, >= 1 */
  int32_t vocab;          /* entries of a row, 1 to 2^20 (else MLA_ERR_UNSUPPORTED) */
  int32_t path_cols;      /* row length of path and tokens_out, >= 1 */
  int64_t target_stride;  /* fp32 elements between rows of target and of draft, >= vocab */
  int64_t draft_stride;
} mla_verify_dims;

/*
 *   target      fp32 [total_q][target_stride], 4-byte aligned (16-byte aligned rows
 *               are read faster): probabilities, in [0, 1] with a sum of about 1
 *               (below 16); a NaN or a value below 0 counts as 0, above 1 as 1
 *   draft       fp32 [total_q][draft_stride], the same, or null: fixed proposals
 *   tokens      int32 [total_q]: the nodes' tokens (that of node 0 is not read).
 *               A node with a token outside [0, vocab) is as if it were not there
 *               (MLA_DEV_BAD_INDEX)
 *   parents     int32 [total_q] as for mla_decode_tree; a node that is not below
 *               node 0 is never reached.  A bad parent: MLA_DEV_BAD_TREE, and the
 *               node is as if it were not there (node 0 stays: it has none)
 *   cu_q_lens   int32 [B + 1] as for mla_prefill, with at most MLA_TREE_MAX_NODES
 *               nodes a request (else MLA_DEV_BAD_QUERY_RANGE, MLA_DEV_BAD_TREE: the
 *               request is treated as one without nodes)
 *   accept      fp32 [total_q]: a random number in [0, 1) per node
 *   sample      fp32 [B]: a random number in [0, 1) per request (in both, others
 *               are taken as the nearest of these, a NaN as 0)
 *   path        int32 [B][path_cols]: node 0 and the accepted nodes, then -1: what
 *               mla_tree_commit takes.  The walk ends where the row is full
 *   tokens_out  int32 [B][path_cols]: the accepted nodes' tokens and the last
 *               token, then -1
 *   num_out     int32 [B]: entries of both; 0 for a request without nodes
 *   status      int32 [1], OR-ed into; the caller clears it
 * The outputs and status overlap neither one another nor the inputs
 * (MLA_ERR_INVALID_ARG; what lies between the rows of target or draft is free).  Rows of target and draft that the walk does not come
 * to are read in single entries only, and may hold anything where no node is.
 */
int mla_verify(const mla_verify_dims* d, const float* target, const float* draft, const int32_t* tokens,
               const int32_t* parents, const int32_t* cu_q_lens, const float* accept, const float* sample,
               int32_t* path, int32_t* tokens_out, int32_t* num_out, int32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_VERIFY_H_ */

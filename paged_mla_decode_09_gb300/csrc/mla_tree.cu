// Entry point mla_decode_tree (see include/mla_tree.h): the chunk attention
// (mla_chunk.cuh, mla_chunk_host.cuh) with the kernels that mask by ancestors.
#include "mla_chunk_host.cuh"
#include "mla_tree.h"

extern "C" {

size_t mla_decode_tree_workspace_size(const mla_prefill_dims* d, int device) {
  return d ? workspace_of<true>(shape_of(d), d->page_size, d->kv_dtype, device) : 0;
}

int mla_decode_tree(const mla_prefill_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                    const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_q_lens,
                    const int32_t* parents, float scale, float kv_scale, void* out, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!d || !cu_q_lens || !parents) return MLA_ERR_INVALID_ARG;
  return run_chunk<true>(shape_of(d), d->page_size, d->kv_dtype, q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens,
                         parents, 0, 0, scale, kv_scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"

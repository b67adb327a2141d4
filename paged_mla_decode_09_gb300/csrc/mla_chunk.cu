// Entry points mla_prefill and mla_decode_window (see include/mla_prefill.h);
// what they share with the tree attention is in mla_chunk_host.cuh.
#include "mla_chunk_host.cuh"
#include "mla_prefill.h"

namespace {

Shape shape_of(const mla_dims* d) {
  Shape s;
  s.B = d->batch; s.H = d->num_heads; s.num_pages = d->num_pages;
  s.T = d->batch >= 1 && d->q_len >= 1 ? static_cast<int64_t>(d->batch) * d->q_len : 0;
  s.max_pages = d->max_pages_per_req; s.stride = d->page_table_stride;
  s.q_len = d->q_len;
  s.f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  return s;
}

}  // namespace

extern "C" {

size_t mla_prefill_workspace_size(const mla_prefill_dims* d, int device) {
  return d ? workspace_of<false>(shape_of(d), d->page_size, d->kv_dtype, device) : 0;
}

int mla_prefill(const mla_prefill_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_q_lens, int32_t window,
                int32_t num_sinks, float scale, float kv_scale, void* out, float* lse, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!d || !cu_q_lens) return MLA_ERR_INVALID_ARG;
  return run_chunk<false>(shape_of(d), d->page_size, d->kv_dtype, q_nope, q_pe, kv_cache, page_table, seq_lens, cu_q_lens,
                          nullptr, window, num_sinks, scale, kv_scale, out, lse, workspace, workspace_bytes, stream);
}

size_t mla_decode_window_workspace_size(const mla_dims* d, int device) {
  return d ? workspace_of<false>(shape_of(d), d->page_size, d->kv_dtype, device) : 0;
}

int mla_decode_window(const mla_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                      const int32_t* page_table, const int32_t* seq_lens, int32_t window, int32_t num_sinks,
                      float scale, float kv_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (!d || window < 1) return MLA_ERR_INVALID_ARG;
  return run_chunk<false>(shape_of(d), d->page_size, d->kv_dtype, q_nope, q_pe, kv_cache, page_table, seq_lens, nullptr,
                          nullptr, window, num_sinks, scale, kv_scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"

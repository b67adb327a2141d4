// Host side shared by the chunk attention's entry points (mla_chunk.cu:
// mla_prefill, mla_decode_window; mla_tree.cu: mla_decode_tree): argument
// checks, workspace layout, tensor maps and the three launches.  kTree selects
// the kernels that mask by the nodes' ancestors; each translation unit
// instantiates its own.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <climits>
#include <cmath>
#include <mutex>

#include "mla_chunk.cuh"
#include "mla_host.h"

namespace {

using mla::chunk::Block;
using mla::chunk::Cfg;
using mla::chunk::Params;

constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per pipeline wait
constexpr int kUncutPages = 3;                  // what the combine's launch costs, in pages

using mla::host::align256;
using mla::host::aligned;
using mla::host::device_ok;
using mla::host::encode_fn;
using mla::host::launch_pdl;
using mla::host::map2;
using mla::host::map3;

// The dimensions both entry points come down to.
struct Shape {
  int64_t B, H, T, num_pages, max_pages, stride;
  int q_len;  // 0: per-request ranges
  bool f8;
  int cg() const;
  int64_t br() const { return 128 * cg(); }
  int64_t blocks() const { return T * H / br() + B; }  // at most: every request ends with a part of a block
};

// Rows per block: 256 (two CTAs per MMA) where a request brings more than 128
// rows on average, else 128.  Measured on GB300: 128 x 2 tokens x 128 heads
// over windows of 2048 (e4m3) 142 us at 256 against 178 at 128; 2 x 512 tokens
// of 128 heads over 8K keys 1279 against 1471; 64 x 64 heads x 1 token over
// windows of 4096, where three quarters of a 256-row block are padding, 125
// against 78.  (Calls with the same rows for every request.  Where one long
// chunk lifts the mean of many short requests, these pad like the last.)
int Shape::cg() const { return T * H > 128 * B ? 2 : 1; }

// [status | blkoff | blocks | prefix | cinfo | cut blocks | partial outputs | partial lse | tree: bad words, ancestors]
struct Layout {
  size_t status, blkoff, blk, prefix, cinfo, cuts, o_part, lse_part, bad, anc, total;
};

template <bool kTree>
Layout layout_of(const Shape& s, int C) {
  Layout l;
  const size_t nb = static_cast<size_t>(s.blocks()), rows = static_cast<size_t>(s.br());
  l.status = 0;
  l.blkoff = 256;
  l.blk = l.blkoff + align256(static_cast<size_t>(s.B + 1) * 4);
  l.prefix = l.blk + align256(nb * sizeof(Block));
  l.cinfo = l.prefix + align256((nb + 1) * 4);
  l.cuts = l.cinfo + align256(static_cast<size_t>(C) * 16);
  l.o_part = l.cuts + align256(static_cast<size_t>(C + 1) * 32);
  l.lse_part = l.o_part + align256(2 * static_cast<size_t>(C) * rows * mla::chunk::kDL * 4);
  l.bad = l.lse_part + align256(2 * static_cast<size_t>(C) * rows * 4);
  l.anc = l.bad + (kTree ? align256(mla::chunk::kTreeBlocks * 4) : 0);
  l.total = l.anc + (kTree ? align256(static_cast<size_t>(s.T) * mla::chunk::kTreeWords * 8) : 0);
  return l;
}

int check_shape(const Shape& s, int page_size, int kv_dtype) {
  if (s.B < 1 || s.H < 1 || s.T < 1 || s.num_pages < 1 || s.max_pages < 1 || s.stride < s.max_pages)
    return MLA_ERR_INVALID_ARG;
  if (page_size != 64) return MLA_ERR_UNSUPPORTED;
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  if (s.T > INT_MAX || s.T * s.H > INT_MAX) return MLA_ERR_UNSUPPORTED;
  if (s.num_pages * 64 > INT_MAX || s.max_pages * 64 > INT_MAX) return MLA_ERR_UNSUPPORTED;
  const int64_t most = s.T * s.H / 128 + s.B;  // blocks
  if (most > 1 << 30 || most * s.max_pages > INT_MAX) return MLA_ERR_UNSUPPORTED;  // the schedule's sums
  return MLA_OK;
}

template <bool kF8, int kCg, bool kTree>
const void* kernel_of() {
  return reinterpret_cast<const void*>(&mla::chunk::mla_chunk_kernel<kF8, kCg, kTree>);
}
template <bool kTree>
const void* kernel_fn(bool f8, int cg) {
  return f8 ? (cg == 2 ? kernel_of<true, 2, kTree>() : kernel_of<true, 1, kTree>())
            : (cg == 2 ? kernel_of<false, 2, kTree>() : kernel_of<false, 1, kTree>());
}
int kernel_smem(bool f8, int cg) {
  return f8 ? (cg == 2 ? Cfg<true, 2>::kSmem : Cfg<true, 1>::kSmem)
            : (cg == 2 ? Cfg<false, 2>::kSmem : Cfg<false, 1>::kSmem);
}

// Clusters of 2 * cg CTAs that run at once (every one gets a slice of the work).
template <bool kTree>
int clusters_of(int device, bool f8, int cg, int* out) {
  static std::mutex mu;
  static int known[64][2][3] = {};
  if (device < 0 || device >= 64) return MLA_ERR_INVALID_ARG;
  std::lock_guard<std::mutex> lk(mu);
  if (known[device][f8][cg]) {
    *out = known[device][f8][cg];
    return MLA_OK;
  }
  int prev = 0;
  if (cudaGetDevice(&prev) != cudaSuccess) return MLA_ERR_CUDA;
  if (prev != device && cudaSetDevice(device) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  int rc = device_ok(device), n = 0;
  if (rc == MLA_OK) {
    const void* fn = kernel_fn<kTree>(f8, cg);
    const int smem = kernel_smem(f8, cg);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * cg * 64, 1, 1);
    cfg.blockDim = dim3(mla::chunk::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * cg;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1)
      rc = MLA_ERR_CUDA;
  }
  if (prev != device) cudaSetDevice(prev);
  if (rc != MLA_OK) {
    cudaGetLastError();
    return rc;
  }
  if (n > mla::chunk::kMaxClusters) n = mla::chunk::kMaxClusters;
  known[device][f8][cg] = n;
  *out = n;
  return MLA_OK;
}

struct Maps {
  CUtensorMap s, o, pe, qn, qp, out, part;
};

// s: an S CTA's part of a page; o: an O CTA's dimensions of a page; pe: the
// e4m3 k_pe rows, or (bf16 pair) single boxes of q_nope; qn, qp: query rows;
// out, part (pairs): where the outputs and the partial ones go.
template <bool kF8, int kCg>
bool make_maps(const void* q_nope, const void* q_pe, const void* kv, const Shape& s, const Params& p, Maps* m) {
  using C = Cfg<kF8, kCg>;
  const int64_t krows = s.num_pages * 64, qrows = s.T * s.H;
  const int row_bytes = kF8 ? 576 : 1152, esz = kF8 ? 1 : 2;
  constexpr bool kPair16 = C::kParts == 3;
  bool ok = map3(&m->s, kv, krows, row_bytes, esz, C::kSBoxes, 64, C::kPartBoxes) &&
            map3(&m->o, kv, krows, row_bytes, esz, C::kSBoxes, 64, kF8 ? C::kRawBoxes : C::kVBoxes) &&
            map3(&m->qn, q_nope, qrows, 1024, 2, 8, C::kQRows, kPair16 ? 3 : 8) &&
            map2(&m->qp, q_pe, qrows, 64, 2, 64, kPair16 ? 128 : C::kQRows, CU_TENSOR_MAP_SWIZZLE_128B);
  m->pe = m->s;
  if (ok && kF8) ok = map2(&m->pe, kv, krows, 576, 1, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B);
  if (ok && kPair16) ok = map2(&m->pe, q_nope, qrows, 512, 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  if (ok) ok = map2(&m->out, p.out, qrows, 512, 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  if (ok)
    ok = map2(&m->part, p.o_part, 2ll * p.C * p.BR, 512, 4, 16, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  return ok;
}

template <bool kF8, int kCg, bool kTree>
cudaError_t launch_attention(const Params& p, const Maps& m, cudaStream_t stream) {
  return launch_pdl(mla::chunk::mla_chunk_kernel<kF8, kCg, kTree>, dim3(2 * kCg * p.C), dim3(mla::chunk::kThreads),
                    Cfg<kF8, kCg>::kSmem, stream, 2 * kCg, p, m.s, m.o, m.pe, m.qn, m.qp, m.out, m.part);
}

template <bool kTree>
int run_chunk(const Shape& s, int page_size, int kv_dtype, const void* q_nope, const void* q_pe, const void* kv_cache,
              const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_q, const int32_t* parents,
              int32_t window, int32_t sinks, float scale, float kv_scale, void* out, float* lse, void* workspace, size_t ws_bytes, void* stream_v) {
  int rc = check_shape(s, page_size, kv_dtype);
  if (rc != MLA_OK) return rc;
  if (!q_nope || !q_pe || !kv_cache || !page_table || !seq_lens || !out || !lse || !workspace)
    return MLA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0) return MLA_ERR_INVALID_ARG;
  if (!mla::host::scale_ok(scale, kv_scale, s.f8)) return MLA_ERR_INVALID_ARG;
  if (!aligned(q_nope, 32) || !aligned(q_pe, 32) || !aligned(kv_cache, 16) || !aligned(out, 32) || !aligned(lse, 4) ||
      !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(parents, 4) ||
      !aligned(workspace, 256))
    return MLA_ERR_ALIGNMENT;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  if ((rc = device_ok(dev)) != MLA_OK) return rc;
  const int cg = s.cg();
  int C = 0;
  if ((rc = clusters_of<kTree>(dev, s.f8, cg, &C)) != MLA_OK) return rc;
  const Layout lay = layout_of<kTree>(s, C);
  if (ws_bytes < lay.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (!encode_fn() || !mla::host::bind_context(dev)) return MLA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Params p;
  p.q_nope = static_cast<const uint8_t*>(q_nope);
  p.q_pe = static_cast<const uint8_t*>(q_pe);
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.o_part = reinterpret_cast<float*>(ws + lay.o_part);
  p.lse_part = reinterpret_cast<float*>(ws + lay.lse_part);
  p.status = reinterpret_cast<int32_t*>(ws + lay.status);
  p.blkoff = reinterpret_cast<int32_t*>(ws + lay.blkoff);
  p.blk = reinterpret_cast<Block*>(ws + lay.blk);
  p.prefix = reinterpret_cast<int32_t*>(ws + lay.prefix);
  p.cinfo = reinterpret_cast<int32_t*>(ws + lay.cinfo);
  p.cuts = reinterpret_cast<int32_t*>(ws + lay.cuts);
  p.parents = parents;
  p.bad = reinterpret_cast<int32_t*>(ws + lay.bad);
  p.anc = reinterpret_cast<uint64_t*>(ws + lay.anc);
  p.B = static_cast<int32_t>(s.B);
  p.H = static_cast<int32_t>(s.H);
  p.q_len = s.q_len;
  p.T = static_cast<int32_t>(s.T);
  p.NB = static_cast<int32_t>(s.blocks());
  p.C = C;
  p.BR = static_cast<int32_t>(s.br());
  p.num_pages = static_cast<int32_t>(s.num_pages);
  p.max_pages = static_cast<int32_t>(s.max_pages);
  p.pt_stride = static_cast<int32_t>(s.stride);
  p.window = window;
  p.sinks = sinks;
  // a piece's start in pages' time: swept on GB300; flat for bf16, an e4m3
  // pair splits its 256 query rows meanwhile (ragged chunks 1477 us at 6, 1427
  // at 10, 1429 at 15, 1459 at 20; two drafts over windows 148, 145, 145, 149;
  // all about 2 % longer since a pair's CTAs order their stores)
  p.unit_cost = s.f8 && cg == 2 ? 15 : 6;
  // what a cut costs, in pages of a cluster's time (~0.75 us): a launch's worth
  // of latency, a block's partials stored by one CTA, all partials written and
  // read.  Measured, one block per cluster against even slices: 1 x 16 heads
  // equal at 5 pages (17.4 us), 1 x 128 at 8, 8 x 64 at 11, 8 x 128 at 15;
  // 64 x 64 heads x 66 pages (56 in even slices) 78 us against 86.  The rule is
  // a line through these points, not measured between them
  const int64_t total_rows = s.T * s.H, rows = total_rows / s.B < p.BR ? total_rows / s.B : p.BR;
  const int64_t whole = 5 + rows / 40 + total_rows / 600;
  p.whole_pages = static_cast<int32_t>(whole < 1000 ? whole : 1000);
  // where no block can have many more pages than that (a window, a short
  // table), none is cut and the combine is left out: 1 x 16 heads over a
  // window of 256 17.5 -> 16.8 us, host 15.0 -> 11.5
  const int64_t tokens = s.T < p.BR / s.H + 2 ? s.T : p.BR / s.H + 2;  // of a block
  int64_t pages = s.max_pages;
  if (window > 0) {
    const int64_t seen = (window + tokens + 62) / 64 + 1 + (static_cast<int64_t>(sinks) + 63) / 64;
    pages = seen < pages ? seen : pages;
  }
  const bool uncut = s.blocks() <= C && pages <= whole + kUncutPages;
  if (uncut) p.whole_pages = INT_MAX / 2;
  p.c2 = mla::host::log2_scale(scale, s.f8 ? kv_scale : 1.f);
  p.kv_scale = s.f8 ? kv_scale : 1.f;
  p.timeout_ns = kTimeoutNs;

  Maps m;
  const bool ok = s.f8 ? (cg == 2 ? make_maps<true, 2>(q_nope, q_pe, kv_cache, s, p, &m)
                                  : make_maps<true, 1>(q_nope, q_pe, kv_cache, s, p, &m))
                       : (cg == 2 ? make_maps<false, 2>(q_nope, q_pe, kv_cache, s, p, &m)
                                  : make_maps<false, 1>(q_nope, q_pe, kv_cache, s, p, &m));
  if (!ok) return MLA_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  using mla::chunk::kSchedSmall;
  // trees: further blocks of the schedule's launch find the nodes' ancestors
  const int64_t tree_blocks = !kTree ? 0 : (s.B < mla::chunk::kTreeBlocks ? s.B : mla::chunk::kTreeBlocks);
  p.tree_blocks = static_cast<int32_t>(tree_blocks);
  const dim3 sched_grid(static_cast<unsigned>(1 + tree_blocks));
  cudaError_t e = s.B <= kSchedSmall && p.NB <= kSchedSmall
                      ? launch_pdl(mla::chunk::mla_chunk_schedule_kernel<true, kTree>, sched_grid, dim3(kSchedSmall), 0,
                                   stream, 0, p)
                      : launch_pdl(mla::chunk::mla_chunk_schedule_kernel<false, kTree>, sched_grid,
                                   dim3(mla::chunk::kSchedThreads), 0, stream, 0, p);
  if (e == cudaSuccess)
    e = s.f8 ? (cg == 2 ? launch_attention<true, 2, kTree>(p, m, stream) : launch_attention<true, 1, kTree>(p, m, stream))
             : (cg == 2 ? launch_attention<false, 2, kTree>(p, m, stream)
                        : launch_attention<false, 1, kTree>(p, m, stream));
  if (e == cudaSuccess && !uncut) {
    // a column per block that may be cut, at most one per slice boundary; a
    // warp per row, or four where that still fits the SMs about once
    const int64_t cuts = s.blocks() < C ? s.blocks() : C;
    const int64_t most = s.T * s.H < p.BR ? s.T * s.H : p.BR;
    const bool four = cuts * most * 4 <= 152 * 32;
    const int64_t items = most * (four ? 4 : 1);
    const dim3 grid(static_cast<unsigned>(cuts),
                    static_cast<unsigned>((items + mla::chunk::kCombineWarps - 1) / mla::chunk::kCombineWarps));
    const dim3 block(mla::chunk::kCombineWarps * 32);
    e = four ? launch_pdl(mla::chunk::mla_chunk_combine_kernel<4, kTree>, grid, block, 0, stream, 0, p)
             : launch_pdl(mla::chunk::mla_chunk_combine_kernel<1, kTree>, grid, block, 0, stream, 0, p);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

Shape shape_of(const mla_prefill_dims* d) {
  Shape s;
  s.B = d->batch; s.H = d->num_heads; s.T = d->total_q; s.num_pages = d->num_pages;
  s.max_pages = d->max_pages_per_req; s.stride = d->page_table_stride;
  s.q_len = 0;
  s.f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  return s;
}
template <bool kTree>
size_t workspace_of(const Shape& s, int page_size, int kv_dtype, int device) {
  if (check_shape(s, page_size, kv_dtype) != MLA_OK) return 0;
  int C = 0;
  if (clusters_of<kTree>(device, s.f8, s.cg(), &C) != MLA_OK) return 0;
  return layout_of<kTree>(s, C).total;
}

}  // namespace

// Page operations (see include/mla_pages.h and mla_tree_commit in
// include/mla_tree.h).
//
// Handing out (mla_page_resize, mla_page_fork): one cluster of eight blocks
// does a call, in steps that a cluster barrier separates: counts copied; pages
// given back or shared (atomic additions: the counts do not depend on their
// order) and missing entries counted; free pages counted; as many free ids as
// entries are missing written to a list, lowest first; the k-th missing entry
// takes the k-th id.  Every block holds a contiguous part of the tables' and of
// the counts' order, so ranks are a block's scan plus the sums of the blocks
// before it.  A free list kept between calls would spare the walk over the
// counts (4 bytes a page), but its order would depend on the calls before.
// What bounds it: the latency of the steps, about four reads and barriers, then
// what eight SMs read.
//
// Rows (mla_tree_commit, mla_page_fork's second kernel): copies of 16-byte
// columns.  A committed path is ascending, so that slot k is read (if at all)
// by a move that is not behind the one that writes it; a thread takes one
// column of the row through all moves in order, eight loads before their
// stores, and needs no barrier.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "mla_host.h"
#include "mla_pages.h"
#include "mla_prefill.h"
#include "mla_sparse.h"
#include "mla_tree.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace pages {

constexpr int kPage = 64;

// ------------------------------------------------------------ handing out
constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 4 * kThreads;  // entries of a step: four in a row per thread

struct Params {
  const int32_t* table;
  const int32_t* refs;
  const int32_t* lens;   // resize: [B] new lengths; fork: [S] the sources'
  const int32_t* src;    // fork: [B]
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* status;
  int32_t* list;         // free ids, as many as entries are missing at most
  int4* copies;          // fork: [B] page, new page (-1: none), rows, -
  int64_t t_stride, o_stride;
  int32_t B, S, cols, P;
};

__device__ __forceinline__ int warp_scan(int v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// The sum of v over the block's threads before this one; `all` over the block.
__device__ __forceinline__ int block_before(int v, int (&warps)[kWarps], int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int incl = warp_scan(v);
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  const int w = warps[lane];
  const int upto = warp_scan(w);
  all = __shfl_sync(0xffffffffu, upto, 31);
  const int base = __shfl_sync(0xffffffffu, upto - w, warp);
  return base + incl - v;
}

// What an entry of the tables is to become.
struct Entry {
  int32_t out;      // kept or shared id, else -1
  bool missing;     // receives a free page
  int32_t change;   // of the count of page `id`
  int32_t id;
  int flag;
  int32_t from, rows;  // fork: the started page and its rows
};

template <bool kFork>
__device__ __forceinline__ Entry entry_at(const Params& p, const int32_t* table, int b, int c) {
  Entry e = {-1, false, 0, 0, 0, -1, 0};
  int s = b;
  if (kFork) {
    s = p.src[b];
    if (s < 0 || s >= p.S) {
      if (s != -1 && c == 0) e.flag = MLA_DEV_BAD_INDEX;
      return e;
    }
  }
  int L = p.lens[s];
  if (L < 0 || L > p.cols * kPage) {
    if (c == 0) e.flag = MLA_DEV_BAD_SEQ_LEN;
    L = L < 0 ? 0 : p.cols * kPage;
  }
  const int need = (L >> 6) + ((L & 63) != 0);
  if (kFork && c >= need) return e;
  const int32_t id = table[static_cast<int64_t>(s) * p.t_stride + c];
  if (kFork) {
    if (id < 0 || id >= p.P) {
      e.flag |= MLA_DEV_BAD_PAGE_ID;
    } else if (c < (L >> 6)) {
      e.out = e.id = id;
      e.change = 1;
    } else {
      e.missing = true;
      e.from = id;
      e.rows = L & 63;
    }
    return e;
  }
  if (id >= p.P) {
    e.flag |= MLA_DEV_BAD_PAGE_ID;
    e.out = c < need ? id : -1;
  } else if (id < 0) {
    e.missing = c < need;
  } else if (c < need) {
    e.out = id;
  } else {
    e.id = id;
    e.change = -1;
  }
  return e;
}

template <bool kFork>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1)
    mla_pages_kernel(const __grid_constant__ Params p) {
  __shared__ int warps[kWarps];
  __shared__ int missing_of[kCluster], free_of[kCluster];  // every block's, written by the blocks themselves
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, rank = static_cast<int>(cluster_ctarank());
  auto tell = [&](int (&dst)[kCluster], int v) {  // v of this block to all
    if (tid < kCluster) st_cluster_u32(mapa(smem_u32(&dst[rank]), static_cast<uint32_t>(tid)), static_cast<uint32_t>(v));
  };
  if (rank == 0 && tid == 0) *p.status = 0;
  if (p.refs_out != p.refs) {
    const bool vec = ((reinterpret_cast<uintptr_t>(p.refs) | reinterpret_cast<uintptr_t>(p.refs_out)) & 15) == 0;
    const int quads = vec ? p.P / 4 : 0, at = rank * kThreads + tid;
    for (int i = at; i < quads; i += kCluster * kThreads)
      reinterpret_cast<int4*>(p.refs_out)[i] = reinterpret_cast<const int4*>(p.refs)[i];
    for (int i = 4 * quads + at; i < p.P; i += kCluster * kThreads) p.refs_out[i] = p.refs[i];
  }
  cluster_sync();  // (also: every block has begun)
  // the tables' entries of this block: [lo, hi) of the rows in one sequence
  const int total = p.B * p.cols;
  const int part = total / kCluster + 1;
  const int lo = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(rank) * part));
  const int hi = total - lo < part ? total : lo + part;
  int missing = 0, flag = 0;
  for (int64_t i0 = lo; i0 < hi; i0 += kTile) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * kThreads + tid;
      if (i >= hi) break;
      const int b = static_cast<int>(i) / p.cols, c = static_cast<int>(i) - b * p.cols;
      const Entry e = entry_at<kFork>(p, p.table, b, c);
      if (kFork && c == 0) p.copies[b] = make_int4(0, -1, 0, 0);
      if (e.change) atomicAdd(p.refs_out + e.id, e.change);
      p.table_out[b * p.o_stride + c] = e.out;
      missing += e.missing;
      flag |= e.flag;
    }
  }
  if (flag) atomicOr(p.status, flag);
  int mine;
  block_before(missing, warps, mine);
  tell(missing_of, mine);
  cluster_sync();
  int wanted = 0, before = 0;  // missing entries in all, and of the blocks before this one
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    wanted += missing_of[r];
    before += r < rank ? missing_of[r] : 0;
  }
  // free pages of this block's part of the counts
  const int ppart = ((p.P + kCluster - 1) / kCluster + 3) & ~3;
  const int plo = static_cast<int>(min(static_cast<int64_t>(p.P), static_cast<int64_t>(rank) * ppart));
  const int phi = p.P - plo < ppart ? p.P : plo + ppart;
  int zeros = 0, below = 0;
  for (int i0 = plo + tid; i0 < phi; i0 += kTile) {
    int v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i0 + u * kThreads < phi ? __ldcg(p.refs_out + i0 + u * kThreads) : 1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (v[u] < 0) {
        p.refs_out[i0 + u * kThreads] = 0;
        below = 1;
      }
      zeros += v[u] <= 0;
    }
  }
  if (below) atomicOr(p.status, MLA_DEV_BAD_REFS);
  if (wanted == 0) return;  // (the same in every block; no block writes to another from here on)
  block_before(zeros, warps, mine);
  tell(free_of, mine);
  cluster_sync();
  int have = 0, fbefore = 0;
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    have += free_of[r];
    fbefore += r < rank ? free_of[r] : 0;
  }
  for (int i0 = plo; i0 < phi && fbefore < wanted; i0 += kTile) {
    int v[4];
    const int i = i0 + 4 * tid;
    int n = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = i + u < phi ? __ldcg(p.refs_out + i + u) : 1;
      n += v[u] <= 0;
    }
    int all;
    int k = fbefore + block_before(n, warps, all);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v[u] <= 0) {
        if (k < wanted) {
          p.list[k] = i + u;
          p.refs_out[i + u] = 1;
        }
        ++k;
      }
    fbefore += all;
  }
  cluster_sync();
  // the k-th missing entry takes the k-th free id
  if (wanted > have && rank == 0 && tid == 0) atomicOr(p.status, MLA_DEV_NO_PAGES);
  if (missing_of[rank] == 0) return;
  for (int64_t i0 = lo; i0 < hi; i0 += kTile) {
    unsigned mask = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + 4 * tid + u;
      if (i >= hi) break;
      const int b = static_cast<int>(i) / p.cols, c = static_cast<int>(i) - b * p.cols;
      // resize: the entry as the first walk left it, which may have been in place
      if (kFork) {
        mask |= entry_at<kFork>(p, p.table, b, c).missing ? 1u << u : 0u;
      } else {
        int L = p.lens[b];
        L = L < 0 ? 0 : (L > p.cols * kPage ? p.cols * kPage : L);
        if (c < (L >> 6) + ((L & 63) != 0) && p.table_out[b * p.o_stride + c] < 0) mask |= 1u << u;
      }
    }
    int all;
    int k = before + block_before(__popc(mask), warps, all);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (mask >> u & 1u) {
        if (k < have) {
          const int64_t i = i0 + 4 * tid + u;
          const int b = static_cast<int>(i) / p.cols, c = static_cast<int>(i) - b * p.cols;
          const int32_t id = __ldcg(p.list + k);
          p.table_out[b * p.o_stride + c] = id;
          if (kFork) {
            const Entry e = entry_at<kFork>(p, p.table, b, c);
            p.copies[b] = make_int4(e.from, id, e.rows, 0);
          }
        }
        ++k;
      }
    before += all;
  }
}

// ------------------------------------------------------------------- rows
constexpr int kCopyThreads = 256;
constexpr int kCopyEach = 6;  // 16-byte columns of a thread: 24 KB a block

// A started page's rows into the child's page: block (child, layer, piece).
__global__ void __launch_bounds__(kCopyThreads)
    mla_pages_copy_kernel(const int4* copies, uint8_t* cache, int64_t layer_stride, int row_bytes) {
  griddep_wait();
  griddep_launch_dependents();
  const int4 c = __ldcg(copies + blockIdx.x);
  const int n = c.z * row_bytes / 16, i0 = blockIdx.z * (kCopyThreads * kCopyEach) + threadIdx.x;
  if (c.y < 0 || i0 >= n) return;
  uint8_t* layer = cache + blockIdx.y * layer_stride;
  const int64_t page = static_cast<int64_t>(kPage) * row_bytes;
  const uint4* src = reinterpret_cast<const uint4*>(layer + c.x * page);
  uint4* dst = reinterpret_cast<uint4*>(layer + c.y * page);
  uint4 v[kCopyEach];
#pragma unroll
  for (int u = 0; u < kCopyEach; ++u)
    if (i0 + u * kCopyThreads < n) v[u] = src[i0 + u * kCopyThreads];
#pragma unroll
  for (int u = 0; u < kCopyEach; ++u)
    if (i0 + u * kCopyThreads < n) dst[i0 + u * kCopyThreads] = v[u];
}

constexpr int kCommitThreads = 288;  // columns of 4 bf16 or 8 e4m3 layers' rows

struct Commit {
  uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu_q;
  const int32_t* path;
  const int32_t* num;
  int32_t* new_lens;
  int32_t* status;
  int64_t layer_stride;
  int32_t cols, num_pages, max_pages, pt_stride, layers, row_bytes;
};

__global__ void __launch_bounds__(kCommitThreads) mla_tree_commit_kernel(const __grid_constant__ Commit p) {
  __shared__ int64_t from[MLA_TREE_MAX_NODES], to[MLA_TREE_MAX_NODES];  // byte offsets of rows; -1: no move
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], L = p.lens[b], a = p.num[b];
  const int64_t nodes = static_cast<int64_t>(q1) - q0;
  int flag = 0;
  if (q0 < 0 || nodes < 0) flag |= MLA_DEV_BAD_QUERY_RANGE;
  else if (nodes > MLA_TREE_MAX_NODES) flag |= MLA_DEV_BAD_TREE;
  else if (L < nodes || L > p.max_pages * kPage) flag |= MLA_DEV_BAD_SEQ_LEN;
  else if (a < 0 || a > nodes || a > p.cols) flag |= MLA_DEV_BAD_INDEX;
  const int n = static_cast<int>(nodes), base = L - n;
  int bad = 0, page_bad = 0;
  if (flag == 0 && tid < a) {
    const int32_t* path = p.path + static_cast<int64_t>(b) * p.cols;
    const int j = path[tid], prev = tid > 0 ? path[tid - 1] : -1;
    bad = j <= prev || j >= n || j < tid;
    int64_t f = -1, t = -1;
    if (!bad && j != tid) {
      const int32_t* row = p.table + static_cast<int64_t>(b) * p.pt_stride;
      const int sf = base + j, st = base + tid;
      const int pf = row[sf / kPage], pt = row[st / kPage];
      if (pf < 0 || pf >= p.num_pages || pt < 0 || pt >= p.num_pages) {
        page_bad = 1;
      } else {
        f = (static_cast<int64_t>(pf) * kPage + sf % kPage) * p.row_bytes;
        t = (static_cast<int64_t>(pt) * kPage + st % kPage) * p.row_bytes;
      }
    }
    from[tid] = f;
    to[tid] = t;
  }
  if (__syncthreads_or(bad)) flag |= MLA_DEV_BAD_INDEX;
  if (blockIdx.x == 0) {
    if (tid == 0) {
      p.new_lens[b] = flag ? L : base + a;
      if (flag) atomicOr(p.status, flag);
    }
    if (!flag && page_bad) atomicOr(p.status, MLA_DEV_BAD_PAGE_ID);
  }
  if (flag) return;
  const int chunks = p.row_bytes / 16;
  const int layer = blockIdx.x * (kCommitThreads / chunks) + tid / chunks;
  if (layer >= p.layers) return;
  uint8_t* col = p.cache + layer * p.layer_stride + (tid % chunks) * 16;
  for (int k0 = 0; k0 < a; k0 += 8) {
    uint4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k0 + u < a && from[k0 + u] >= 0) v[u] = *reinterpret_cast<const uint4*>(col + from[k0 + u]);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (k0 + u < a && from[k0 + u] >= 0) *reinterpret_cast<uint4*>(col + to[k0 + u]) = v[u];
  }
}

}  // namespace pages
}  // namespace mla

namespace {

using mla::host::align256;
using mla::host::aligned;
using mla::host::launch_pdl;

int current_device_ok() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return mla::host::device_ok(dev);
}

// Whether two int32 tables share an element, counted from first to last.
bool overlap(const int32_t* a, int64_t an, const int32_t* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + 4 * static_cast<uintptr_t>(bn) && y < x + 4 * static_cast<uintptr_t>(an);
}
int64_t extent(int64_t rows, int64_t stride, int64_t cols) { return (rows - 1) * stride + cols; }

bool sizes_ok(int64_t rows, int64_t cols, int64_t pages) {
  return cols * 64 <= INT_MAX && rows * cols <= INT_MAX && pages <= 1 << 30;
}

// [status | free ids | copies]
size_t list_bytes(int64_t rows, int64_t cols, int64_t pages) {
  return align256(4 * static_cast<size_t>(rows * cols < pages ? rows * cols : pages));
}
int64_t cache_bytes(int64_t num_pages, bool f8) { return num_pages * 64 * (f8 ? 576 : 1152); }

template <bool kFork>
cudaError_t launch(const mla::pages::Params& p, cudaStream_t s) {
  return launch_pdl(&mla::pages::mla_pages_kernel<kFork>, dim3(mla::pages::kCluster), dim3(mla::pages::kThreads), 0, s, 0,
                    p);
}

}  // namespace

extern "C" {

size_t mla_page_resize_workspace_size(int32_t batch, int32_t max_pages_per_req, int32_t num_pages) {
  if (batch < 1 || max_pages_per_req < 1 || num_pages < 1 || !sizes_ok(batch, max_pages_per_req, num_pages)) return 0;
  return 256 + list_bytes(batch, max_pages_per_req, num_pages);
}

int mla_page_resize(const mla_page_resize_dims* d, const int32_t* new_lens, const int32_t* page_table,
                    const int32_t* page_refs, int32_t* page_table_out, int32_t* page_refs_out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!d || !new_lens || !page_table || !page_refs || !page_table_out || !page_refs_out || !workspace)
    return MLA_ERR_INVALID_ARG;
  const int64_t B = d->batch, cols = d->max_pages_per_req, P = d->num_pages;
  if (B < 1 || P < 1 || cols < 1 || d->table_stride < cols || d->out_stride < cols) return MLA_ERR_INVALID_ARG;
  if (!sizes_ok(B, cols, P)) return MLA_ERR_UNSUPPORTED;
  if (!aligned(new_lens, 4) || !aligned(page_table, 4) || !aligned(page_refs, 4) || !aligned(page_table_out, 4) ||
      !aligned(page_refs_out, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGNMENT;
  const bool in_place = page_table == page_table_out && d->table_stride == d->out_stride;
  if (!in_place && overlap(page_table, extent(B, d->table_stride, cols), page_table_out, extent(B, d->out_stride, cols)))
    return MLA_ERR_INVALID_ARG;
  if (page_refs != page_refs_out && overlap(page_refs, P, page_refs_out, P)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < mla_page_resize_workspace_size(d->batch, d->max_pages_per_req, d->num_pages))
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  const int rc = current_device_ok();
  if (rc != MLA_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  mla::pages::Params p = {};
  p.table = page_table;
  p.refs = page_refs;
  p.lens = new_lens;
  p.table_out = page_table_out;
  p.refs_out = page_refs_out;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.list = reinterpret_cast<int32_t*>(ws + 256);
  p.t_stride = d->table_stride;
  p.o_stride = d->out_stride;
  p.B = p.S = d->batch;
  p.cols = d->max_pages_per_req;
  p.P = d->num_pages;
  if (launch<false>(p, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

size_t mla_page_fork_workspace_size(int32_t sources, int32_t children, int32_t max_pages_per_req, int32_t num_pages) {
  if (sources < 1 || children < 1 || max_pages_per_req < 1 || num_pages < 1 ||
      !sizes_ok(children, max_pages_per_req, num_pages))
    return 0;
  return 256 + list_bytes(children, 1, num_pages) + align256(static_cast<size_t>(children) * 16);
}

int mla_page_fork(const mla_page_fork_dims* d, const int32_t* src, const int32_t* seq_lens, const int32_t* page_table,
                  const int32_t* page_refs, void* kv_cache, int32_t* page_table_out, int32_t* page_refs_out,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (!d || !src || !seq_lens || !page_table || !page_refs || !kv_cache || !page_table_out || !page_refs_out || !workspace)
    return MLA_ERR_INVALID_ARG;
  const int64_t S = d->sources, B = d->children, cols = d->max_pages_per_req, P = d->num_pages;
  if (S < 1 || B < 1 || d->num_layers < 1 || P < 1 || cols < 1 || d->table_stride < cols || d->out_stride < cols)
    return MLA_ERR_INVALID_ARG;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  const bool f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  if (!sizes_ok(B, cols, P) || d->num_layers > 65535 || P * 64 > INT_MAX) return MLA_ERR_UNSUPPORTED;
  if (d->num_layers > 1 && d->layer_stride < cache_bytes(P, f8)) return MLA_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) || !aligned(page_refs, 4) ||
      !aligned(kv_cache, 16) || !aligned(page_table_out, 4) || !aligned(page_refs_out, 4) || !aligned(workspace, 256) ||
      (d->num_layers > 1 && d->layer_stride % 16 != 0))
    return MLA_ERR_ALIGNMENT;
  if (overlap(page_table, extent(S, d->table_stride, cols), page_table_out, extent(B, d->out_stride, cols)))
    return MLA_ERR_INVALID_ARG;
  if (page_refs != page_refs_out && overlap(page_refs, P, page_refs_out, P)) return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < mla_page_fork_workspace_size(d->sources, d->children, d->max_pages_per_req, d->num_pages))
    return MLA_ERR_WORKSPACE_TOO_SMALL;
  const int rc = current_device_ok();
  if (rc != MLA_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  mla::pages::Params p = {};
  p.table = page_table;
  p.refs = page_refs;
  p.lens = seq_lens;
  p.src = src;
  p.table_out = page_table_out;
  p.refs_out = page_refs_out;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.list = reinterpret_cast<int32_t*>(ws + 256);
  p.copies = reinterpret_cast<int4*>(ws + 256 + list_bytes(B, 1, P));
  p.t_stride = d->table_stride;
  p.o_stride = d->out_stride;
  p.B = d->children;
  p.S = d->sources;
  p.cols = d->max_pages_per_req;
  p.P = d->num_pages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch<true>(p, s);
  if (e == cudaSuccess) {
    using namespace mla::pages;
    const int row = f8 ? 576 : 1152, piece = kCopyThreads * kCopyEach * 16;
    const dim3 grid(static_cast<unsigned>(B), static_cast<unsigned>(d->num_layers),
                    static_cast<unsigned>((63 * row + piece - 1) / piece));
    e = launch_pdl(&mla_pages_copy_kernel, grid, dim3(kCopyThreads), 0, s, 0, static_cast<const int4*>(p.copies),
                   static_cast<uint8_t*>(kv_cache), d->num_layers > 1 ? d->layer_stride : static_cast<int64_t>(0), row);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

int mla_tree_commit(const mla_tree_commit_dims* d, void* kv_cache, const int32_t* page_table, const int32_t* seq_lens,
                    const int32_t* cu_q_lens, const int32_t* path, const int32_t* num_path, int32_t* new_lens,
                    int32_t* status, void* stream) {
  if (!d || !kv_cache || !page_table || !seq_lens || !cu_q_lens || !path || !num_path || !new_lens || !status)
    return MLA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_layers < 1 || d->path_cols < 1 || d->num_pages < 1 || d->max_pages_per_req < 1 ||
      d->page_table_stride < d->max_pages_per_req)
    return MLA_ERR_INVALID_ARG;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  const bool f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  if (d->batch > 65535 || d->num_layers > 65535 || static_cast<int64_t>(d->max_pages_per_req) * 64 > INT_MAX ||
      static_cast<int64_t>(d->num_pages) * 64 > INT_MAX)
    return MLA_ERR_UNSUPPORTED;
  if (d->num_layers > 1 && d->layer_stride < cache_bytes(d->num_pages, f8)) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q_lens, 4) ||
      !aligned(path, 4) || !aligned(num_path, 4) || !aligned(new_lens, 4) || !aligned(status, 4) ||
      (d->num_layers > 1 && d->layer_stride % 16 != 0))
    return MLA_ERR_ALIGNMENT;
  if (overlap(seq_lens, d->batch, new_lens, d->batch)) return MLA_ERR_INVALID_ARG;
  const int rc = current_device_ok();
  if (rc != MLA_OK) return rc;
  using namespace mla::pages;
  Commit p = {};
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.table = page_table;
  p.lens = seq_lens;
  p.cu_q = cu_q_lens;
  p.path = path;
  p.num = num_path;
  p.new_lens = new_lens;
  p.status = status;
  p.layer_stride = d->num_layers > 1 ? d->layer_stride : 0;
  p.cols = d->path_cols;
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages_per_req;
  p.pt_stride = d->page_table_stride;
  p.layers = d->num_layers;
  p.row_bytes = f8 ? 576 : 1152;
  const int per = kCommitThreads / (p.row_bytes / 16);
  const dim3 grid(static_cast<unsigned>((d->num_layers + per - 1) / per), static_cast<unsigned>(d->batch));
  if (launch_pdl(&mla_tree_commit_kernel, grid, dim3(kCommitThreads), 0, static_cast<cudaStream_t>(stream), 0, p) !=
      cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // extern "C"

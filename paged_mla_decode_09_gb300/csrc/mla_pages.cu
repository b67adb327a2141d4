// Page operations (see include/mla_pages.h and mla_tree_commit in
// include/mla_tree.h).
//
// Handing out (mla_page_resize, mla_page_fork): one block or a cluster of up
// to 16 does a call, in steps that a cluster barrier separates: counts copied and
// their zeros counted; pages given back or shared (atomic additions: the counts
// do not depend on their order; what becomes free is added to its block's
// zeros) and each row's missing entries counted; as many free ids as entries
// are missing written to a list, lowest first; the k-th missing entry takes the
// k-th id.  Every block holds a contiguous part of the rows and of the counts,
// so ranks are a block's scan plus the sums of the blocks before it, and blocks
// behind the last id that is wanted have nothing to list.  A free list kept
// between calls would spare the walk over the counts (4 bytes a page), but its
// order would depend on the calls before.
// What bounds it: the latency of the steps, about four reads and barriers, then
// what 16 SMs read: 4 requests over 512 pages 3.0 us, 256 requests of 512 columns
// over 131072 pages 12.0 (counts 1.3, their barrier 0.9, entries and the slowest
// block's atomics 4.4, sums 0.9, the list 1.6, the entries' pages 1.6).  Times
// in this file: a call of a graph of calls.
//
// Rows (mla_tree_commit, mla_page_fork's second kernel): copies of 16-byte
// columns.  A committed path is ascending, so that slot k is read (if at all)
// by a move that is not behind the one that writes it; a thread takes one
// column of the row through all moves in order, eight loads before their
// stores, and needs no barrier.  64 requests in 24 layers 3.3 us (4.6 MB, 1.4
// TB/s: the launch and three dependent reads), 64 forks in 16 layers 11.6 with
// the handing out (35 MB).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <initializer_list>
#include <mutex>

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
template <bool kFork>
constexpr int kOneBlock = kFork ? 10240 : 16384;  // entries and pages up to which one block does a call (see launch)
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 4 * kThreads;  // pages of a step: four in a row per thread

struct Params {
  const int32_t* table;
  const int32_t* refs;
  const int32_t* lens;   // resize: [B] new lengths; fork: [S] the sources'
  const int32_t* src;    // fork: [B]
  int32_t* table_out;
  int32_t* refs_out;
  int32_t* status;
  int32_t* missing;      // [B] entries of each row that receive a free page
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

__device__ __forceinline__ void red_cluster_add(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// What a row of the output is made of: `row` of the input, its first `keep`
// entries as they are (fork: shared), the entries below `need` present, those
// from there on not.  fork: need - keep is 1 where a page has been started.
struct Row {
  const int32_t* row;
  int keep, need, tail, flag;
};

template <bool kFork>
__device__ __forceinline__ Row row_of(const Params& p, int b) {
  Row r = {p.table, 0, 0, 0, 0};
  int s = b;
  if (kFork) {
    s = p.src[b];
    if (s < 0 || s >= p.S) {
      if (s != -1) r.flag = MLA_DEV_BAD_INDEX;
      return r;
    }
  }
  int L = p.lens[s];
  if (L < 0 || L > p.cols * kPage) {
    r.flag = MLA_DEV_BAD_SEQ_LEN;
    L = L < 0 ? 0 : p.cols * kPage;
  }
  r.row = p.table + s * p.t_stride;
  r.keep = L >> 6;
  r.tail = L & 63;
  r.need = r.keep + (r.tail != 0);
  if (!kFork) r.keep = r.need;
  return r;
}

template <int kCluster>
__device__ __forceinline__ void sync_all() {
  if constexpr (kCluster == 1) __syncthreads();
  else cluster_sync();
}

template <bool kFork, int kCluster>
__global__ void __launch_bounds__(kThreads, 1) mla_pages_kernel(const __grid_constant__ Params p) {
  __shared__ int warps[kWarps];
  __shared__ int missing_of[kCluster];  // every block's, written by the blocks themselves
  __shared__ int free_of[kCluster];
  __shared__ int free_pages;            // of this block's part of the counts
  __shared__ int lacks[kThreads], begins[kThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = kCluster == 1 ? 0 : static_cast<int>(cluster_ctarank());
  if (rank == 0 && tid == 0) *p.status = 0;
  // rows of the tables: a contiguous part of them per block
  const int rpart = static_cast<int>((static_cast<int64_t>(p.B) + kCluster - 1) / kCluster);
  const int rlo = static_cast<int>(min(static_cast<int64_t>(p.B), static_cast<int64_t>(rank) * rpart));
  const int rhi = p.B - rlo < rpart ? p.B : rlo + rpart;
  for (int b = rlo + tid; b < rhi; b += kThreads) p.missing[b] = 0;
  // this block's part of the counts: copied, at least 0, free pages counted
  const int ppart = (p.P / kCluster + 4) & ~3;
  const int plo = static_cast<int>(min(static_cast<int64_t>(p.P), static_cast<int64_t>(rank) * ppart));
  const int phi = p.P - plo < ppart ? p.P : plo + ppart;
  const bool vec = ((reinterpret_cast<uintptr_t>(p.refs) | reinterpret_cast<uintptr_t>(p.refs_out)) & 15) == 0;
  int zeros = 0, below = 0, all;
  {
    const bool copy = p.refs_out != p.refs;
    const int quads = vec ? (phi - plo) / 4 : 0;
    const int4* src = reinterpret_cast<const int4*>(p.refs + plo);
    int4* dst = reinterpret_cast<int4*>(p.refs_out + plo);
#pragma unroll 4
    for (int i = tid; i < quads; i += kThreads) {
      int4 v = src[i];
      const bool neg = (v.x | v.y | v.z | v.w) < 0;
      if (neg) {
        v = make_int4(max(v.x, 0), max(v.y, 0), max(v.z, 0), max(v.w, 0));
        below = 1;
      }
      zeros += (v.x == 0) + (v.y == 0) + (v.z == 0) + (v.w == 0);
      if (copy || neg) dst[i] = v;
    }
    for (int i = plo + 4 * quads + tid; i < phi; i += kThreads) {
      const int v = p.refs[i];
      if (copy || v < 0) p.refs_out[i] = max(v, 0);
      below |= v < 0;
      zeros += v <= 0;
    }
  }
  block_before(zeros, warps, all);
  if (tid == 0) free_pages = all;
  sync_all<kCluster>();  // every block has begun, the counts are in place, the status is clear
  if (below) atomicOr(p.status, MLA_DEV_BAD_REFS);
  // entries, four of a row a time: kFly times four of them in flight
  auto owner = [&](int id) { return mapa(smem_u32(&free_pages), static_cast<uint32_t>(id / ppart)); };
  constexpr int kFly = 2;
  const uint32_t per_row = static_cast<uint32_t>(p.cols + 3) / 4, quads = static_cast<uint32_t>(rhi - rlo) * per_row;
  const bool tvec = ((reinterpret_cast<uintptr_t>(p.table) | 4 * p.t_stride) & 15) == 0;
  const bool ovec = ((reinterpret_cast<uintptr_t>(p.table_out) | 4 * p.o_stride) & 15) == 0;
  int lacking = 0, flag = 0;
  for (uint32_t i0 = tid; i0 < quads; i0 += kFly * kThreads) {
    Row r[kFly];
    int b[kFly], c[kFly];
    int32_t id[kFly][4];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const uint32_t i = i0 + f * kThreads, row = i < quads ? i / per_row : 0;
      b[f] = rlo + static_cast<int>(row);
      c[f] = i < quads ? 4 * static_cast<int>(i - row * per_row) : p.cols;
      if (!kFork && c[f] < p.cols) {  // (does not wait for the length)
        const int32_t* at = p.table + b[f] * p.t_stride + c[f];
        if (tvec && c[f] + 4 <= p.cols) {
          const int4 v = *reinterpret_cast<const int4*>(at);
          id[f][0] = v.x; id[f][1] = v.y; id[f][2] = v.z; id[f][3] = v.w;
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u) id[f][u] = c[f] + u < p.cols ? at[u] : -1;
        }
      }
      if (c[f] < p.cols) r[f] = row_of<kFork>(p, b[f]);
    }
    if (kFork)
#pragma unroll
      for (int f = 0; f < kFly; ++f)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c[f] < p.cols) id[f][u] = c[f] + u < r[f].need ? r[f].row[c[f] + u] : -1;
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      if (c[f] >= p.cols) break;
      int32_t o[4];
      int missing = 0, old[4];
      unsigned did = 0;  // entries whose page's count changed
      flag |= r[f].flag;
      // (the page that has been started, if any: the new one is added below)
      const int started = r[f].keep - c[f];
      if (kFork && (r[f].tail == 0 ? c[f] == 0 : started >= 0 && started < 4)) {
        int e = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) e = u == started ? id[f][u] : e;
        p.copies[b[f]] = make_int4(e, -1, r[f].tail, r[f].keep);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = c[f] + u, e = id[f][u];
        o[u] = -1;
        if (kFork) {
          if (col >= r[f].need) continue;
          if (e < 0 || e >= p.P) {
            flag |= MLA_DEV_BAD_PAGE_ID;
          } else if (col < r[f].keep) {
            o[u] = e;
            old[u] = atomicAdd(p.refs_out + e, 1);
            did |= 1u << u;
          } else {
            ++missing;
          }
        } else {
          if (e >= p.P) flag |= MLA_DEV_BAD_PAGE_ID;
          if (col >= p.cols) continue;
          if (col < r[f].need) {
            o[u] = e < 0 ? -1 : e;
            missing += e < 0;
          } else if (e >= 0 && e < p.P) {  // given back
            old[u] = atomicSub(p.refs_out + e, 1);
            did |= 1u << u;
          }
        }
      }
      int32_t* out = p.table_out + b[f] * p.o_stride + c[f];
      if (ovec && c[f] + 4 <= p.cols) {
        *reinterpret_cast<int4*>(out) = make_int4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c[f] + u < p.cols) out[u] = o[u];
      }
      if (missing) atomicAdd(p.missing + b[f], missing);
      lacking += missing;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = id[f][u];
        if (!(did >> u & 1u)) continue;
        if (kFork) {
          if (old[u] == 0) red_cluster_add(owner(e), -1);  // (a count that was wrong)
        } else if (old[u] == 1) {  // free now
          red_cluster_add(owner(e), 1);
        } else if (old[u] <= 0) {  // given back more often than it was named: the count stays 0
          atomicAdd(p.refs_out + e, 1);
          flag |= MLA_DEV_BAD_REFS;
        }
      }
    }
  }
  if (flag) atomicOr(p.status, flag);
  block_before(lacking, warps, all);
  if (tid < kCluster)
    st_cluster_u32(mapa(smem_u32(&missing_of[rank]), static_cast<uint32_t>(tid)), static_cast<uint32_t>(all));
  sync_all<kCluster>();
  int wanted = 0, before = 0;  // missing entries in all, and of the blocks before this one
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    wanted += missing_of[r];
    before += r < rank ? missing_of[r] : 0;
  }
  if (wanted == 0) return;  // (the same in every block, before any reads another's shared memory)
  // free pages of all blocks, read where they are counted: no block ends before the next barrier
  if (tid < kCluster)
    free_of[tid] = static_cast<int>(ld_cluster_u32(mapa(smem_u32(&free_pages), static_cast<uint32_t>(tid))));
  __syncthreads();
  int have = 0, fbefore = 0;
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    have += free_of[r];
    fbefore += r < rank ? free_of[r] : 0;
  }
  // the lowest free ids
  for (int i0 = plo; i0 < phi && fbefore < wanted; i0 += kTile) {
    int v[4];
    const int i = i0 + 4 * tid;
    int n = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[u] = i + u < phi ? __ldcg(p.refs_out + i + u) : 1;
      n += v[u] <= 0;
    }
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
  sync_all<kCluster>();
  // the k-th missing entry takes the k-th free id
  if (wanted > have && rank == 0 && tid == 0) atomicOr(p.status, MLA_DEV_NO_PAGES);
  if (missing_of[rank] == 0) return;
  for (int b0 = rlo; b0 < rhi; b0 += kThreads) {
    const int b = b0 + tid, n = b < rhi ? __ldcg(p.missing + b) : 0;
    const int at = before + block_before(n, warps, all);  // where the row's entries begin in the list
    before += all;
    if (kFork) {  // the one entry behind the shared ones
      if (n > 0 && at < have) {
        const int4 c = p.copies[b];
        const int32_t id = __ldcg(p.list + at);
        p.copies[b] = make_int4(c.x, id, c.z, 0);
        p.table_out[b * p.o_stride + c.w] = id;
      }
      continue;
    }
    lacks[tid] = n;
    begins[tid] = at;
    __syncthreads();
    for (int j = warp; j < kThreads && b0 + j < rhi; j += kWarps) {  // a warp per row, from its end, where requests grow
      if (lacks[j] == 0) continue;
      int L = p.lens[b0 + j];
      L = L > p.cols * kPage ? p.cols * kPage : L;
      const int need = (L >> 6) + ((L & 63) != 0), k = begins[j];
      int32_t* out = p.table_out + (b0 + j) * p.o_stride;
      int upto = k + lacks[j];
      for (int c0 = (need - 1) / 32 * 32; c0 >= 0 && upto > k; c0 -= 32) {
        const int c = c0 + lane;
        const unsigned lack = __ballot_sync(0xffffffffu, c < need && out[c] < 0);
        upto -= __popc(lack);
        const int place = upto + __popc(lack & ((1u << lane) - 1u));
        if ((lack >> lane & 1u) && place < have) out[c] = __ldcg(p.list + place);
      }
    }
    __syncthreads();
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
  int64_t f = -1, t = -1;
  if (flag == 0 && tid < a) {
    const int32_t* path = p.path + static_cast<int64_t>(b) * p.cols;
    const int j = path[tid], prev = tid > 0 ? path[tid - 1] : -1;
    bad = j <= prev || j >= n || j < tid;
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
  }
  if (tid < MLA_TREE_MAX_NODES) {
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
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
  return mla::host::overlap(a, 4 * an, b, 4 * bn);
}
int64_t extent(int64_t rows, int64_t stride, int64_t cols) { return (rows - 1) * stride + cols; }

struct Table {
  const int32_t* at;
  int64_t rows, stride;
};
struct Vec {
  const int32_t* at;
  int64_t n;
};
// Whether an output of a page call (table, counts) or its workspace shares
// memory with another buffer; table over table and counts over counts apart,
// which have rules of their own.  Blocks read all of them in every step.
bool outputs_overlap(const Table& table, const Table& out, int64_t cols, const int32_t* refs, const int32_t* refs_out,
                     int64_t pages, const void* workspace, size_t bytes, std::initializer_list<Vec> inputs) {
  const int64_t words = static_cast<int64_t>(bytes / 4);
  auto in_table = [&](const Table& t, const void* v, int64_t n) {
    return mla::host::overlap_rows(t.at, t.rows, t.stride, cols, v, n);
  };
  for (const Vec& v : inputs)
    if (in_table(out, v.at, v.n) || overlap(refs_out, pages, v.at, v.n) || overlap(workspace, words, v.at, v.n)) return true;
  return in_table(out, refs, pages) || in_table(out, refs_out, pages) || in_table(table, refs_out, pages) ||
         in_table(out, workspace, words) || in_table(table, workspace, words) ||
         overlap(workspace, words, refs, pages) || overlap(workspace, words, refs_out, pages);
}

bool sizes_ok(int64_t rows, int64_t cols, int64_t pages) {
  return cols * 64 <= INT_MAX && rows * cols <= INT_MAX && pages <= 1 << 30;
}

// [status | missing entries of each row | free ids | copies]
size_t list_bytes(int64_t rows, int64_t cols, int64_t pages) {
  return align256(4 * static_cast<size_t>(rows * cols < pages ? rows * cols : pages));
}
size_t row_bytes(int64_t rows) { return align256(4 * static_cast<size_t>(rows)); }
int64_t cache_bytes(int64_t num_pages, bool f8) { return num_pages * 64 * (f8 ? 576 : 1152); }

// Whether clusters of 16 blocks (beyond the portable 8) fit on the device.
template <bool kFork>
bool sixteen_fit(int device) {
  static std::mutex mu;
  static int8_t known[64] = {};  // 1: they do, 2: they do not
  if (device < 0 || device >= 64) return false;
  std::lock_guard<std::mutex> lk(mu);
  if (!known[device]) {
    const void* fn = reinterpret_cast<const void*>(&mla::pages::mla_pages_kernel<kFork, 16>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(mla::pages::kThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool ok = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                    cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess && n >= 1;
    if (!ok) cudaGetLastError();
    known[device] = ok ? 1 : 2;
  }
  return known[device] == 1;
}

// One block for small calls (its barriers are cheaper), else a cluster of 16
// where that fits.  Measured, one block and a cluster, us a call of a graph:
//   resize, entries and pages  6.1K 5.4, 7.3   12.3K 6.0, 8.0   16.4K 7.2, 8.3
//                              32.8K 11.0, 8.9   65.5K 17.2, 9.3   262K 46.5, 12.7
//     with 8 entries only      6K 3.3, 3.7   12K 3.7, 3.7   16K 4.0, 3.7   40K 5.9, 3.9
//   fork (with its copies)     4.9K 8.5, 11.1   8.2K 11.0, 11.9   12.5K 12.6, 11.5
//                              25.7K 19.4, 11.9
// (a cluster of 8 took 14.1 where 16 blocks took 11.7).
template <bool kFork>
cudaError_t launch(const mla::pages::Params& p, cudaStream_t s) {
  using namespace mla::pages;
  const dim3 block(kThreads);
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (static_cast<int64_t>(p.B) * p.cols + p.P > kOneBlock<kFork> && sixteen_fit<kFork>(dev))
    return launch_pdl(&mla_pages_kernel<kFork, 16>, dim3(16), block, 0, s, 16, p);
  return launch_pdl(&mla_pages_kernel<kFork, 1>, dim3(1), block, 0, s, 0, p);
}

}  // namespace

extern "C" {

size_t mla_page_resize_workspace_size(int32_t batch, int32_t max_pages_per_req, int32_t num_pages) {
  if (batch < 1 || max_pages_per_req < 1 || num_pages < 1 || !sizes_ok(batch, max_pages_per_req, num_pages)) return 0;
  return 256 + row_bytes(batch) + list_bytes(batch, max_pages_per_req, num_pages);
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
  const size_t need = mla_page_resize_workspace_size(d->batch, d->max_pages_per_req, d->num_pages);
  if (outputs_overlap({page_table, B, d->table_stride}, {page_table_out, B, d->out_stride}, cols, page_refs, page_refs_out,
                      P, workspace, need, {{new_lens, B}}))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
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
  p.missing = reinterpret_cast<int32_t*>(ws + 256);
  p.list = reinterpret_cast<int32_t*>(ws + 256 + row_bytes(B));
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
  return 256 + row_bytes(children) + list_bytes(children, 1, num_pages) + align256(static_cast<size_t>(children) * 16);
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
  const size_t need = mla_page_fork_workspace_size(d->sources, d->children, d->max_pages_per_req, d->num_pages);
  if (outputs_overlap({page_table, S, d->table_stride}, {page_table_out, B, d->out_stride}, cols, page_refs, page_refs_out,
                      P, workspace, need, {{src, B}, {seq_lens, S}}))
    return MLA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
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
  p.missing = reinterpret_cast<int32_t*>(ws + 256);
  p.list = reinterpret_cast<int32_t*>(ws + 256 + row_bytes(B));
  p.copies = reinterpret_cast<int4*>(ws + 256 + row_bytes(B) + list_bytes(B, 1, P));
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
  // every layer's block of a request reads the inputs, the first one writes the outputs
  const int64_t B = d->batch;
  for (const Vec& out : {Vec{new_lens, B}, Vec{status, 1}}) {
    for (const Vec& in : {Vec{seq_lens, B}, Vec{cu_q_lens, B + 1}, Vec{num_path, B}, Vec{path, B * d->path_cols}})
      if (overlap(in.at, in.n, out.at, out.n)) return MLA_ERR_INVALID_ARG;
    if (mla::host::overlap_rows(page_table, B, d->page_table_stride, d->max_pages_per_req, out.at, out.n))
      return MLA_ERR_INVALID_ARG;
  }
  if (overlap(new_lens, B, status, 1)) return MLA_ERR_INVALID_ARG;
  if (!aligned(kv_cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_q_lens, 4) ||
      !aligned(path, 4) || !aligned(num_path, 4) || !aligned(new_lens, 4) || !aligned(status, 4) ||
      (d->num_layers > 1 && d->layer_stride % 16 != 0))
    return MLA_ERR_ALIGNMENT;
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

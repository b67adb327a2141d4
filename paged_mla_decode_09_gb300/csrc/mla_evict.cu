// mla_evict (see include/mla_evict.h): which tokens a request keeps, and the
// rows that move.
//
// Selection (one block per request): the k-th greatest of L 32-bit keys by
// radix selection (11 + 11 + 10 bits, a shared-memory histogram each), then
// one ordered walk that ranks the ties by slot and lists the free slots below
// k and the kept tokens behind.  Firm tokens have the greatest key, so one
// rule covers them.  The keys live in shared memory where they fit (48K
// tokens), else they are formed again from the inputs on every walk.
//
// Moves: a kept token below k stays, so only the tokens kept behind k move,
// each into a place that no kept token uses: sources and destinations are
// disjoint and all rows copy at once, without a staging buffer.  (Compacting
// in order instead would move nearly every row behind the first dropped one:
// for 4096 of 4224 tokens about 4000 rows of a request instead of 125.)
//
// What bounds it: at a few hundred KB per request the latency of the walks
// (a dozen barriers and the loads of L keys per 1024 threads), then the moved
// rows' bytes.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "mla_evict.h"
#include "mla_host.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace evict {

constexpr int kPage = 64;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxSmemKeys = 48 * 1024;

struct Params {
  const float* mass;
  const int32_t* positions;
  const int32_t* seq_lens;
  const int32_t* page_table;
  uint8_t* cache;
  int32_t* new_lens;
  int32_t* kept;
  float* mass_out;
  int32_t* positions_out;
  int32_t* status;
  int32_t* counts;   // [B] moves; -1 - moves where the length was bad
  int32_t* movers;   // [B][budget] old slots of the tokens that move
  int32_t* holes;    // [B][budget] the slots that receive them
  int32_t B, cols, cap, num_pages, pt_stride, budget, sinks, recent, smem_keys;
};

// Keys that order like the weights: a NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the block's earlier warps of a per-warp value; total in *all.
__device__ __forceinline__ int warps_before(int mine, int* buf, int* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) buf[warp] = mine;
  __syncthreads();
  const int v = buf[lane];  // 32 warps
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  *all = __shfl_sync(0xffffffffu, s, 31);
  return __shfl_sync(0xffffffffu, s - v, warp);
}

__global__ void __launch_bounds__(kThreads) mla_evict_select_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kBins];
  __shared__ int buf[kWarps];
  __shared__ int pick[2];  // the digit of the k-th key, keys above it
  griddep_launch_dependents();
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (b == 0 && tid < 4) p.status[tid] = 0;
  const int Lraw = p.seq_lens[b];
  const bool bad = Lraw < 0 || Lraw > p.cap;
  const int L = Lraw < 0 ? 0 : (Lraw > p.cap ? p.cap : Lraw);
  const int k = L < p.budget ? L : p.budget;
  const float* mass = p.mass + static_cast<int64_t>(b) * p.cols;
  const int32_t* pos = p.positions ? p.positions + static_cast<int64_t>(b) * p.cols : nullptr;
  float* mass_out = p.mass_out + static_cast<int64_t>(b) * p.cols;
  int32_t* pos_out = pos ? p.positions_out + static_cast<int64_t>(b) * p.cols : nullptr;
  int32_t* kept = p.kept + static_cast<int64_t>(b) * p.budget;
  int32_t* movers = p.movers + static_cast<int64_t>(b) * p.budget;
  int32_t* holes = p.holes + static_cast<int64_t>(b) * p.budget;
  int moves = 0;
  if (k < L) {
    // the greatest position
    int last = L - 1;
    if (pos) {
      int m = -1;
      for (int t = tid; t < L; t += kThreads) m = max(m, pos[t]);
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) buf[warp] = m;
      __syncthreads();
      last = __reduce_max_sync(0xffffffffu, buf[lane]);
      __syncthreads();
    }
    const int64_t firm_from = static_cast<int64_t>(last) - p.recent + 1;
    auto form = [&](int t) -> uint32_t {
      const int q = pos ? pos[t] : t;
      return (q < p.sinks || q >= firm_from) ? 0xFFFFFFFFu : weight_key(mass[t]);
    };
    const bool cached = L <= p.smem_keys;
    if (cached) {
      for (int t = tid; t < L; t += kThreads) keys[t] = form(t);
    }
    auto key = [&](int t) -> uint32_t { return cached ? keys[t] : form(t); };
    // radix selection of the k-th greatest key
    uint32_t prefix = 0, mask = 0;
    int need = k;  // rank within the keys that share the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const int bins = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < bins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int t = tid; t < L; t += kThreads) {
        const uint32_t x = key(t);
        if ((x & mask) == prefix) atomicAdd(&hist[(x >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // from the greatest digit down: thread i has bins [lo, lo + per), the
      // warps' sums in that order
      const int per = bins / kThreads;
      const int top = bins - 1 - tid * per;
      int c[2];
      c[0] = hist[top];
      c[1] = per == 2 ? hist[top - 1] : 0;
      int s = c[0] + c[1];
      const int own = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      int all;
      const int before = warps_before(__shfl_sync(0xffffffffu, s, 31), buf, &all) + s - own;
      if (before < need && before + own >= need) {  // one thread
        const bool second = before + c[0] < need;
        pick[0] = second ? top - 1 : top;
        pick[1] = before + (second ? c[0] : 0);
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      need -= pick[1];
      __syncthreads();
    }
    // keys above prefix are kept, and of the keys equal to it the `need`
    // lowest slots.  Each warp walks a contiguous range of slots.
    const int per_warp = ((L + kWarps - 1) / kWarps + 31) & ~31;
    const int t0 = warp * per_warp, t1 = min(L, t0 + per_warp);
    int ties = 0;
    for (int t = t0 + lane; t - lane < t1; t += 32)
      ties += __popc(__ballot_sync(0xffffffffu, t < t1 && key(t) == prefix));
    int all;
    const int tie0 = warps_before(ties, buf, &all);
    // free slots below k and movers behind it, counted, then written in order
    int nh = 0, nm = 0, tie = tie0;
    for (int t = t0 + lane; t - lane < t1; t += 32) {
      const bool in = t < t1;
      const uint32_t x = in ? key(t) : 0u;
      const unsigned eq = __ballot_sync(0xffffffffu, in && x == prefix);
      const bool keep = in && (x > prefix || (x == prefix && tie + __popc(eq & ((1u << lane) - 1u)) < need));
      tie += __popc(eq);
      nh += __popc(__ballot_sync(0xffffffffu, in && t < k && !keep));
      nm += __popc(__ballot_sync(0xffffffffu, in && t >= k && keep));
    }
    int h = warps_before(nh, buf, &all);
    int m = warps_before(nm, buf, &moves);
    tie = tie0;
    for (int t = t0 + lane; t - lane < t1; t += 32) {
      const bool in = t < t1;
      const uint32_t x = in ? key(t) : 0u;
      const unsigned below = (1u << lane) - 1u;
      const unsigned eq = __ballot_sync(0xffffffffu, in && x == prefix);
      const bool keep = in && (x > prefix || (x == prefix && tie + __popc(eq & below) < need));
      tie += __popc(eq);
      const unsigned hb = __ballot_sync(0xffffffffu, in && t < k && !keep);
      const unsigned mb = __ballot_sync(0xffffffffu, in && t >= k && keep);
      if (in && t < k && !keep) holes[h + __popc(hb & below)] = t;
      if (in && t >= k && keep) movers[m + __popc(mb & below)] = t;
      if (in && t < k && keep) kept[t] = t;
      h += __popc(hb);
      m += __popc(mb);
    }
    __syncthreads();
    // outputs: only slots below k are written and only slots that stay below
    // k or movers from k on are read, so outputs may be the inputs
    for (int j = tid; j < moves; j += kThreads) {
      const int t = holes[j], o = movers[j];
      kept[t] = o;
      mass_out[t] = mass[o];
      if (pos) pos_out[t] = pos[o];
    }
    __syncthreads();
    for (int t = tid; t < k; t += kThreads) {
      if (kept[t] != t) continue;
      mass_out[t] = mass[t];
      if (pos) pos_out[t] = pos[t];
    }
  } else {
    for (int t = tid; t < k; t += kThreads) {
      kept[t] = t;
      mass_out[t] = mass[t];
      if (pos) pos_out[t] = pos[t];
    }
  }
  for (int t = k + tid; t < p.budget; t += kThreads) kept[t] = -1;
  if (tid == 0) {
    p.new_lens[b] = k;
    p.counts[b] = bad ? -1 - moves : moves;
  }
}

// Rows [blockIdx.x .. step gridDim.x) of request blockIdx.y's moves, one warp
// per row, all of its loads first.
constexpr int kMoveWarps = 8;

template <int kRowBytes>
__global__ void __launch_bounds__(kMoveWarps * 32) mla_evict_move_kernel(const __grid_constant__ Params p) {
  constexpr int kChunks = kRowBytes / 16;
  constexpr int kPer = (kChunks + 31) / 32;
  griddep_wait();
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int n0 = p.counts[b];
  const int n = n0 < 0 ? -1 - n0 : n0;
  if (n0 < 0 && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.status, MLA_DEV_BAD_SEQ_LEN);
  const int32_t* movers = p.movers + static_cast<int64_t>(b) * p.budget;
  const int32_t* holes = p.holes + static_cast<int64_t>(b) * p.budget;
  const int32_t* table = p.page_table + static_cast<int64_t>(b) * p.pt_stride;
  for (int j = blockIdx.x * kMoveWarps + (threadIdx.x >> 5); j < n; j += gridDim.x * kMoveWarps) {
    const int from = movers[j], to = holes[j];
    const int pf = table[from / kPage], pt = table[to / kPage];
    if (pf < 0 || pf >= p.num_pages || pt < 0 || pt >= p.num_pages) {
      if (lane == 0) atomicOr(p.status, MLA_DEV_BAD_PAGE_ID);
      continue;
    }
    const uint4* src =
        reinterpret_cast<const uint4*>(p.cache + (static_cast<int64_t>(pf) * kPage + from % kPage) * kRowBytes);
    uint4* dst = reinterpret_cast<uint4*>(p.cache + (static_cast<int64_t>(pt) * kPage + to % kPage) * kRowBytes);
    uint4 v[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (lane + 32 * q < kChunks) v[q] = src[lane + 32 * q];
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (lane + 32 * q < kChunks) dst[lane + 32 * q] = v[q];
  }
}

}  // namespace evict
}  // namespace mla

namespace {

using mla::evict::Params;
using namespace mla::host;

struct Layout {
  size_t counts, movers, holes, total;
};
Layout layout_of(int64_t B, int64_t budget) {
  Layout l;
  l.counts = 256;
  l.movers = l.counts + align256(static_cast<size_t>(B) * 4);
  l.holes = l.movers + align256(static_cast<size_t>(B * budget) * 4);
  l.total = l.holes + align256(static_cast<size_t>(B * budget) * 4);
  return l;
}

}  // namespace

extern "C" {

size_t mla_evict_workspace_size(int32_t batch, int32_t budget) {
  return batch < 1 || budget < 1 ? 0 : layout_of(batch, budget).total;
}

int mla_evict(const mla_evict_dims* d, const float* mass, const int32_t* positions, const int32_t* seq_lens,
              const int32_t* page_table, void* kv_cache, int32_t* new_lens, int32_t* kept, float* mass_out,
              int32_t* positions_out, void* workspace, size_t workspace_bytes, void* stream_v) {
  if (!d || d->batch < 1 || d->mass_cols < 1 || d->num_pages < 1 || d->max_pages_per_req < 1 ||
      d->page_table_stride < d->max_pages_per_req || d->budget < 1 || d->num_sinks < 0 || d->num_recent < 0 ||
      static_cast<int64_t>(d->num_sinks) + d->num_recent > d->budget)
    return MLA_ERR_INVALID_ARG;
  if (!mass || !seq_lens || !page_table || !kv_cache || !new_lens || !kept || !mass_out || !workspace ||
      (positions && !positions_out))
    return MLA_ERR_INVALID_ARG;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(d->num_pages) * 64 > INT_MAX || static_cast<int64_t>(d->max_pages_per_req) * 64 > INT_MAX ||
      d->batch > 65535)  // the move grid's y extent
    return MLA_ERR_UNSUPPORTED;
  if (!aligned(mass, 4) || !aligned(positions, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) ||
      !aligned(kv_cache, 16) || !aligned(new_lens, 4) || !aligned(kept, 4) || !aligned(mass_out, 4) ||
      !aligned(positions_out, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGNMENT;
  const Layout lay = layout_of(d->batch, d->budget);
  if (workspace_bytes < lay.total) return MLA_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0, rc, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  if ((rc = device_ok(dev)) != MLA_OK) return rc;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return MLA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Params p;
  p.mass = mass;
  p.positions = positions;
  p.seq_lens = seq_lens;
  p.page_table = page_table;
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.new_lens = new_lens;
  p.kept = kept;
  p.mass_out = mass_out;
  p.positions_out = positions_out;
  p.status = reinterpret_cast<int32_t*>(ws);
  p.counts = reinterpret_cast<int32_t*>(ws + lay.counts);
  p.movers = reinterpret_cast<int32_t*>(ws + lay.movers);
  p.holes = reinterpret_cast<int32_t*>(ws + lay.holes);
  p.B = d->batch;
  p.cols = d->mass_cols;
  p.cap = d->max_pages_per_req * 64 < d->mass_cols ? d->max_pages_per_req * 64 : d->mass_cols;
  p.num_pages = d->num_pages;
  p.pt_stride = d->page_table_stride;
  p.budget = d->budget;
  p.sinks = d->num_sinks;
  p.recent = d->num_recent;
  p.smem_keys = p.cap < mla::evict::kMaxSmemKeys ? p.cap : mla::evict::kMaxSmemKeys;
  const int smem = ((p.smem_keys * 4) + 15) & ~15;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  cudaError_t e = allow_smem<0>(mla::evict::mla_evict_select_kernel, mla::evict::kMaxSmemKeys * 4, dev);
  if (e == cudaSuccess) {
    mla::evict::mla_evict_select_kernel<<<d->batch, mla::evict::kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    // about eight blocks per SM in all, each request's rows over its share
    const int rows = mla::evict::kMoveWarps;
    const int64_t most = (static_cast<int64_t>(d->budget) + rows - 1) / rows;
    int64_t gx = (8ll * sms + d->batch - 1) / d->batch;
    if (gx > most) gx = most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(d->batch), 1);
    cfg.blockDim = dim3(mla::evict::kMoveWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = d->kv_dtype == MLA_KV_FP8_E4M3 ? cudaLaunchKernelEx(&cfg, mla::evict::mla_evict_move_kernel<576>, p)
                                       : cudaLaunchKernelEx(&cfg, mla::evict::mla_evict_move_kernel<1152>, p);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // extern "C"

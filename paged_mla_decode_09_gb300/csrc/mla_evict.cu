// mla_evict (see include/mla_evict.h): which tokens a request keeps, and the
// rows that move.
//
// Selection (a cluster of 1 to 8 blocks per request, each with a contiguous
// part of the slots): the k-th greatest of L 32-bit keys by radix selection
// (four digits of 8 bits: every block counts its digits in shared memory and
// adds up all blocks' counts over distributed shared memory, 256 words a
// block and digit; with 2048 bins those reads took 4 us a digit), then one
// walk that counts and one that ranks the ties by slot and lists the free
// slots below k and the kept tokens behind.  Firm tokens have the greatest
// key, so one rule covers them.  The keys live in shared memory where they fit
// (20K tokens a block), else they are formed again from the inputs on every
// walk.  512 threads, so that two blocks share an SM: clusters of 8 blocks of
// 1024 threads did not all fit at once (16 requests ran in two waves).
//
// Moves: a kept token below k stays, so only the tokens kept behind k move,
// each into a place that no kept token uses: sources and destinations are
// disjoint and all rows copy at once, without a staging buffer.  (Compacting
// in order instead would move nearly every row behind the first dropped one:
// for 4096 of 4224 tokens about 4000 rows of a request instead of 125.)
//
// What bounds it: the latency of about a dozen walks and barriers (a block per
// request took 59 us for 16 requests of up to 32K tokens, clusters take 28), then
// the moved rows' bytes.  64 requests of 4.2K tokens take 15.5 us, one of 600
// 7.7.  (The moves by the selecting blocks themselves took 3 to 9 us longer: a
// launch of their own finds its blocks resident already and spreads the rows
// over every SM.)
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "mla_evict.h"
#include "mla_host.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace evict {

constexpr int kPage = 64;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 256;
constexpr int kMaxSmemKeys = 20 * 1024;  // 8 bytes a token: key and position

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
  int32_t cluster;   // blocks per request
};

// Keys that order like the weights: a NaN lowest, -0 equal to 0.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads, 2) mla_evict_select_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint32_t keys[];  // keys of the block's slots, then their positions
  __shared__ int hist[4][kBins];
  __shared__ int buf[kWarps];
  __shared__ int pick[3];          // the digit of the k-th key, keys above it, whether all keys of it are kept
  __shared__ uint32_t lim[4][2];   // least and greatest of a pass's keys
  __shared__ uint32_t lims[2];     // the same over the cluster
  __shared__ int4 counts_w[kWarps];  // per warp, see below
  __shared__ int4 share;           // the block's sums of them, and its greatest position: read by the other blocks
  __shared__ int share_pos;
  griddep_wait();
  griddep_launch_dependents();
  const int cs = p.cluster, b = blockIdx.x / cs, rank = blockIdx.x % cs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0 && tid < 4) p.status[tid] = 0;
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
  const int step = cs * kThreads, first = rank * kThreads + tid;  // shares of the copies below
  auto sync_ranks = [&]() {
    if (cs > 1) cluster_sync();
    else __syncthreads();
  };
  if (k < L) {  // the same in every block of the cluster
    const int part = ((L + cs - 1) / cs + 31) & ~31;  // slots of a block
    const int r0 = rank * part < L ? rank * part : L, r1 = r0 + part < L ? r0 + part : L;
    const bool cached = part <= p.smem_keys;
    int32_t* spos = reinterpret_cast<int32_t*>(keys) + p.smem_keys;
    for (int i = tid; i < 4 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
    if (tid < 8) lim[tid >> 1][tid & 1] = tid & 1 ? 0u : 0xFFFFFFFFu;
    int last = L - 1;  // the greatest position
    {
      // Every slot below k gets its own weight and position back, also those
      // that a mover takes over below: the values are at hand, and a later walk
      // would wait for each of them (the outputs may be the inputs).
      int m = -1;
      constexpr int kFly = 8;
      for (int t = r0 + tid; t < r1; t += kFly * kThreads) {  // 16 loads in flight
        int qv[kFly];
        float xv[kFly];
#pragma unroll
        for (int q = 0; q < kFly; ++q) {
          const int at = t + q * kThreads;
          qv[q] = pos && at < r1 ? pos[at] : -1;
          xv[q] = at < r1 && (cached || at < k) ? mass[at] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < kFly; ++q) {
          const int at = t + q * kThreads;
          if (at >= r1) break;
          m = max(m, qv[q]);
          if (cached) {
            keys[at - r0] = weight_key(xv[q]);
            if (pos) spos[at - r0] = qv[q];
          }
          if (at < k) {
            mass_out[at] = xv[q];
            if (pos) pos_out[at] = qv[q];
          }
        }
      }
      if (pos) {
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == 0) buf[warp] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, buf[lane % kWarps]);
        if (tid == 0) share_pos = m;
        sync_ranks();
        last = -1;
        for (int r = 0; r < cs; ++r) last = max(last, static_cast<int>(ld_cluster_u32(mapa(smem_u32(&share_pos), r))));
      } else {
        __syncthreads();
      }
    }
    const int64_t firm_from = static_cast<int64_t>(last) - p.recent + 1;
    auto firm = [&](int q) { return q < p.sinks || q >= firm_from; };
    // the key of slot t (0 past the block's slots); the first walk makes it
    // final in shared memory
    auto form = [&](int t) -> uint32_t {
      if (t >= r1) return 0u;
      if (cached) return firm(pos ? spos[t - r0] : t) ? 0xFFFFFFFFu : keys[t - r0];
      return firm(pos ? pos[t] : t) ? 0xFFFFFFFFu : weight_key(mass[t]);
    };
    // radix selection of the k-th greatest key
    uint32_t prefix = 0, mask = 0;
    int need = k;  // rank within the keys that share the prefix
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      uint32_t least = 0xFFFFFFFFu, most = 0u;
      for (int t = r0 + tid; t - lane < r1; t += kThreads) {
        uint32_t x;
        if (pass == 0 || !cached) {
          x = form(t);
          if (cached && t < r1) keys[t - r0] = x;
        } else {
          x = t < r1 ? keys[t - r0] : 0u;
        }
        const bool in = t < r1 && (x & mask) == prefix;
        if (in) {
          atomicAdd(&hist[pass][(x >> shift) & 255u], 1);
          least = min(least, x);
          most = max(most, x);
        }
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) {
        atomicMin(&lim[pass][0], least);
        atomicMax(&lim[pass][1], most);
      }
      sync_ranks();
      // from the greatest digit down: thread i has bin 255 - i of all blocks
      int own = 0;
      if (tid < kBins) {
        const uint32_t at = smem_u32(&hist[pass][kBins - 1 - tid]);
        uint32_t c[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) c[r] = r < cs ? ld_cluster_u32(mapa(at, r)) : 0u;
#pragma unroll
        for (int r = 0; r < 8; ++r) own += static_cast<int>(c[r]);
      } else if (warp == kBins / 32) {  // lanes r and 8 + r: block r's least and greatest key
        const int r = lane & 7, w = lane >> 3 & 1;
        const uint32_t x = r < cs ? ld_cluster_u32(mapa(smem_u32(&lim[pass][w]), r)) : (w ? 0u : 0xFFFFFFFFu);
        const uint32_t a = __reduce_min_sync(0xffffffffu, w ? 0xFFFFFFFFu : x);
        const uint32_t b = __reduce_max_sync(0xffffffffu, w ? x : 0u);
        if (lane == 0) {
          lims[0] = a;
          lims[1] = b;
        }
      }
      int sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
      }
      if (lane == 31) buf[warp] = sum;
      __syncthreads();
      int before = sum - own;
      for (int w = 0; w < warp && w < kBins / 32; ++w) before += buf[w];
      if (tid < kBins && before < need && before + own >= need) {  // one thread
        pick[0] = kBins - 1 - tid;
        pick[1] = before;
        pick[2] = before + own == need;
      }
      __syncthreads();
      if (lims[0] == lims[1]) {  // equal keys (tokens never attended to, say): that is the k-th, ties by slot
        prefix = lims[0];
        break;
      }
      prefix |= static_cast<uint32_t>(pick[0]) << shift;
      mask |= 255u << shift;
      need -= pick[1];
      if (pick[2]) {  // the keys from prefix on are the k (not all L, so prefix is not 0): no ties, no more digits
        prefix -= 1;
        need = 0;
        break;
      }
    }
    auto key = [&](int t) -> uint32_t { return cached ? (t < r1 ? keys[t - r0] : 0u) : form(t); };
    // Keys above prefix are kept, and of the keys equal to it the `need`
    // lowest slots.  Each warp walks a contiguous range of the block's slots
    // and counts (x) ties below k, (y) ties from k on, (z) slots below k with a
    // smaller key or a tie, (w) greater keys from k on; how many of its ties
    // are kept follows from the ties before it, and with it its free slots
    // below k and its movers.
    const int per_warp = ((r1 - r0 + kWarps - 1) / kWarps + 31) & ~31;
    const int t0 = min(r1, r0 + warp * per_warp), t1 = min(r1, t0 + per_warp);
    int4 n = make_int4(0, 0, 0, 0);
    for (int t = t0 + lane; t - lane < t1; t += 32) {
      const bool in = t < t1;
      const uint32_t x = in ? key(t) : 0u;
      n.x += __popc(__ballot_sync(0xffffffffu, in && t < k && x == prefix));
      n.y += __popc(__ballot_sync(0xffffffffu, in && t >= k && x == prefix));
      n.z += __popc(__ballot_sync(0xffffffffu, in && t < k && x <= prefix));
      n.w += __popc(__ballot_sync(0xffffffffu, in && t >= k && x > prefix));
    }
    if (lane == 0) counts_w[warp] = n;
    __syncthreads();
    if (tid == 0) {
      int4 a = make_int4(0, 0, 0, 0);
      for (int w = 0; w < kWarps; ++w) {
        a.x += counts_w[w].x; a.y += counts_w[w].y; a.z += counts_w[w].z; a.w += counts_w[w].w;
      }
      share = a;
    }
    sync_ranks();
    // Free slots and movers of the blocks and warps before this warp: lane i
    // has part i (a block, then a warp of this block); `need` less the ties
    // before it says how many of its ties are kept, and scans add up the rest.
    int tie = 0, h = 0, m = 0;
    auto scan = [&](int v) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
      }
      return v;
    };
    // adds the parts before part `at` to (tie, h, m); the last lane's sums in all[]
    int all_m = 0;
    auto add_before = [&](int4 c, int at) {
      const int ties = scan(c.x + c.y), before = tie + ties - (c.x + c.y);
      const int lo = min(max(need - before, 0), c.x);        // kept ties below k
      const int hi = min(max(need - before - c.x, 0), c.y);  // and from k on
      const int hs = scan(c.z - lo), ms = scan(c.w + hi);
      all_m = m + __shfl_sync(0xffffffffu, ms, 15);
      const int src = at > 0 ? at - 1 : 0;
      const int t1 = __shfl_sync(0xffffffffu, ties, src), h1 = __shfl_sync(0xffffffffu, hs, src),
                m1 = __shfl_sync(0xffffffffu, ms, src);
      if (at > 0) {
        tie += t1;
        h += h1;
        m += m1;
      }
    };
    int4 c = make_int4(0, 0, 0, 0);
    if (lane < cs) {
      const uint32_t at = mapa(smem_u32(&share), lane);
      c = make_int4(static_cast<int>(ld_cluster_u32(at)), static_cast<int>(ld_cluster_u32(at + 4)),
                    static_cast<int>(ld_cluster_u32(at + 8)), static_cast<int>(ld_cluster_u32(at + 12)));
    }
    add_before(c, rank);
    moves = all_m;
    c = lane < kWarps ? counts_w[lane] : make_int4(0, 0, 0, 0);
    add_before(c, warp);
    const unsigned below = (1u << lane) - 1u;
    for (int t = t0 + lane; t - lane < t1; t += 32) {
      const bool in = t < t1;
      const uint32_t x = in ? key(t) : 0u;
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
    sync_ranks();  // the lists are whole, every key has been read, and no block reads another's memory any more
    // only slots below k are written, only ones from k on are read
    for (int j = first; j < moves; j += step) {
      const int t = holes[j], o = movers[j];
      kept[t] = o;
      mass_out[t] = mass[o];
      if (pos) pos_out[t] = pos[o];
    }
  } else {
    for (int t = first; t < k; t += step) {
      kept[t] = t;
      mass_out[t] = mass[t];
      if (pos) pos_out[t] = pos[t];
    }
  }
  for (int t = k + first; t < p.budget; t += step) kept[t] = -1;
  if (rank == 0 && tid == 0) {
    p.new_lens[b] = k;
    p.counts[b] = bad ? -1 - moves : moves;
  }
}

// Rows [blockIdx.x .. step gridDim.x) of request blockIdx.y's moves, one warp
// per row, all of its loads first (four rows a warp took 1 to 1.5 us longer:
// a quarter of the warps).
constexpr int kMoveWarps = 8;

template <int kRowBytes>
__global__ void __launch_bounds__(kMoveWarps * 32) mla_evict_move_kernel(const __grid_constant__ Params p) {
  constexpr int kChunks = kRowBytes / 16;
  constexpr int kPer = (kChunks + 31) / 32;
  griddep_wait();
  griddep_launch_dependents();
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

constexpr int kMaxTokens = 1 << 30;  // a walk's slot and step then stay within int32

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
      d->mass_cols > kMaxTokens || d->budget > kMaxTokens || d->batch > 65535)  // the move grid's y extent
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
  // blocks per request: as many as fit two to an SM, each with 512 slots or
  // more (a thread's worth each)
  p.cluster = 1;
  while (p.cluster < 8 && p.cluster * static_cast<int64_t>(d->batch) <= sms &&
         p.cap / (2 * p.cluster) >= mla::evict::kThreads)
    p.cluster *= 2;
  const int part = ((p.cap + p.cluster - 1) / p.cluster + 31) & ~31;
  p.smem_keys = part < mla::evict::kMaxSmemKeys ? part : mla::evict::kMaxSmemKeys;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  cudaError_t e = allow_smem<0>(mla::evict::mla_evict_select_kernel, mla::evict::kMaxSmemKeys * 8, dev);
  if (e == cudaSuccess) {
    e = launch_pdl(mla::evict::mla_evict_select_kernel, dim3(static_cast<unsigned>(d->batch) * p.cluster),
                   dim3(mla::evict::kThreads), static_cast<size_t>(p.smem_keys) * 8, stream, p.cluster, p);
  }
  if (e == cudaSuccess) {
    // about eight blocks per SM in all, each request's rows over its share
    const int rows = mla::evict::kMoveWarps;
    const int64_t most = (static_cast<int64_t>(d->budget) + rows - 1) / rows;
    int64_t gx = (8ll * sms + d->batch - 1) / d->batch;
    if (gx > most) gx = most;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(d->batch)), block(mla::evict::kMoveWarps * 32);
    e = d->kv_dtype == MLA_KV_FP8_E4M3 ? launch_pdl(mla::evict::mla_evict_move_kernel<576>, grid, block, 0, stream, 0, p)
                                       : launch_pdl(mla::evict::mla_evict_move_kernel<1152>, grid, block, 0, stream, 0, p);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // extern "C"

// mla_attn_mass (see include/mla_evict.h): the softmax weight that a step's
// queries gave to every cached token.
//
//     mass_out[t] = mass[t] + sum_r 2^(s_rt c - lse_r log2e),
//
// r over the request's query rows (positions x heads).  The scores are
// computed again (1152 flops per row and key, and every cache row read once),
// which needs no store of the attention's weights.
//
// Two kernels, by which operand is the smaller one:
//
//   * at most 128 query rows per request (decode steps): the queries stay in
//     tensor memory and the pages stream by (lane = query row).  Each CTA takes
//     a slice of all pages.  Per page two groups of four warps (even and odd
//     pages) take exp2, each warp adds its 32 rows by halving exchanges (62
//     shuffles leave every lane the sums of two keys) and 64 threads add the
//     four warps' sums to the keys' values.  Bound by HBM: 72 KB per page and
//     CTA are ~3100 cycles of its share, against 1224 tensor cycles: 64 x 64
//     heads over 8K keys 97 us, 6.4 TB/s.
//   * more rows (a prompt's last tokens): 128 keys stay in tensor memory (an
//     e4m3 cache's expanded to bf16, which is exact) and the query rows stream
//     by, 64 at a time (lane = key), so that a key's sum is a thread's own
//     running sum: no exchanges, every cache row read once, and the bf16
//     queries need no splitting.  Bound by the tensor pipe: 36 MMAs of 34
//     cycles per 128 keys x 64 rows.  (With the queries kept instead, every
//     CTA moved and split all row blocks for the few pages of its slice: 503
//     us for 32 tokens x 128 heads over 75K keys of four requests, e4m3; this
//     way 192, the pipe 87 % busy.)
//     Where a call has few key tiles, a cluster of 2 to 8 CTAs shares one,
//     every CTA some of the row tiles, and the first adds up their sums.
//
// No atomics: a key belongs to one CTA, or to one cluster whose first CTA adds
// up the others' sums, in a fixed order either way, so results do not depend
// on timing or slicing.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <mutex>

#include "mla_evict.h"
#include "mla_host.h"
#include "mla_mass_plan.h"
#include "mla_score.cuh"

namespace mla {
namespace mass {

using chunk::kDL;
using chunk::kLog2e;
using chunk::kPage;
using chunk::kRows;
using chunk::kThreads;

constexpr int kUnitCost = 4;  // pages' worth of starting a piece

template <bool kF8>
struct Lay {
  using C = chunk::Cfg<kF8, 1>;
  static constexpr int kSums = C::kNStS * C::kSlotS;  // [group][2][4 warps][64] column sums
  static constexpr int kData = kSums + 2 * 2 * 4 * 64 * 4;
  static constexpr int kSmem = 1024 + kData + 512;
  static_assert(kSmem <= 232448, "shared memory budget");
};

struct __align__(8) Ctrl {
  uint64_t kv_full[chunk::kMaxStages];
  uint64_t kv_empty[chunk::kMaxStages];
  uint64_t q_bar[2];
  uint64_t s_full[6];  // mla_mass_kernel: 3
  uint64_t s_empty[3];
  uint64_t q_full;
  uint64_t sums[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int first;          // first request of this CTA's slice
  long long start;    // its weighted start
  long long total;    // weighted length of all requests
};
static_assert(sizeof(Ctrl) <= 512, "control block");

struct Params {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* lse;
  const float* mass_in;
  float* mass_out;
  int32_t* status;
  int32_t B, H, Q, R;
  int32_t num_pages, max_pages, pt_stride, cols;
  int32_t cap;        // longest length the table and the mass rows hold
  int32_t num_fresh;
  int32_t cluster;    // CTAs that share a key tile (the first kernel: 1)
  float c2;           // scale log2(e) (kv_scale), rounded once
  uint64_t timeout_ns;
};

__global__ void mla_mass_clear_kernel(int32_t* status) {
  griddep_wait();  // before the kernel behind it may read its inputs
  griddep_launch_dependents();
  if (threadIdx.x < 4) status[threadIdx.x] = 0;
}

__device__ __forceinline__ int length_of(const Params& p, int b) {
  const int L = p.seq_lens[b];
  return L < 0 ? 0 : (L > p.cap ? p.cap : L);
}

// The pieces of requests in a CTA's slice, in order.
struct Unit {
  int b, L, p0, p1;
};
struct UnitIter {
  const Params* p;
  long long x0, x1, start;
  int b;
  __device__ void init(const Params& pp, const Ctrl* c) {
    p = &pp;
    x0 = c->total * blockIdx.x / gridDim.x;
    x1 = c->total * (blockIdx.x + 1) / gridDim.x;
    start = c->start;
    b = c->first;
  }
  __device__ bool next(Unit& u) {
    while (b < p->B && start < x1) {
      u.b = b;
      u.L = length_of(*p, b);
      const int np = (u.L + kPage - 1) / kPage;
      const long long lo = x0 - start - kUnitCost, hi = x1 - start - kUnitCost;
      u.p0 = lo > 0 ? (lo < np ? static_cast<int>(lo) : np) : 0;
      u.p1 = hi < np ? (hi > 0 ? static_cast<int>(hi) : 0) : np;
      start += kUnitCost + np;
      ++b;
      if (u.p0 < u.p1) return true;
    }
    return false;
  }
};

enum WaitTag : int { kWaitEmpty = 201, kWaitOther, kWaitLanded, kWaitQFull, kWaitSPrev, kWaitQ, kWaitS, kWaitSums };

__device__ __forceinline__ void raise_timeout(const Params& p, Ctrl* ctrl, int tag, uint32_t j) {
  if (atomicCAS(p.status + 1, 0, tag) == 0) {
    p.status[2] = static_cast<int32_t>(j);
    p.status[3] = static_cast<int32_t>((blockIdx.x << 16) | (threadIdx.x >> 5));
  }
  atomicOr(p.status, MLA_DEV_TIMEOUT);
  *reinterpret_cast<volatile int*>(&ctrl->abort) = 1;
}

// Where this CTA's slice of a line begins on which request b occupies
// weight(length of b): two passes over the lengths (inputs of the call, so
// before griddep_wait), first the total, then the request that holds the
// slice's start.  All threads; returns whether this thread saw a bad length.
template <typename Weight>
__device__ __forceinline__ bool find_slice(const Params& p, Ctrl* ctrl, Weight weight) {
  __shared__ long long wsum[kThreads / 32];
  __shared__ long long carry;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = false;
  for (int pass = 0; pass < 2; ++pass) {
    if (tid == 0) carry = 0;
    __syncthreads();
    const long long x0 = pass ? ctrl->total * (blockIdx.x / p.cluster) / (gridDim.x / p.cluster) : 0;
    for (int base = 0; base < p.B; base += kThreads) {
      const int b = base + tid;
      long long v = 0;
      if (b < p.B) {
        // through L2: a line of an earlier call may sit in this SM's L1 until griddep_wait
        const int L = __ldcg(p.seq_lens + b);
        bad = bad || L < p.Q || L > p.cap;
        v = weight(L < 0 ? 0 : (L > p.cap ? p.cap : L));
      }
      const long long own = v;
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
      }
      if (lane == 31) wsum[warp] = v;
      __syncthreads();
      long long before = carry;
      for (int w = 0; w < warp; ++w) before += wsum[w];
      const long long end = before + v;
      if (pass && b < p.B && end > x0 && end - own <= x0) {  // exactly one request
        ctrl->first = b;
        ctrl->start = end - own;
      }
      __syncthreads();
      if (tid == kThreads - 1) carry = end;
      __syncthreads();
    }
    if (tid == 0 && !pass) ctrl->total = carry;
    __syncthreads();
  }
  return bad;
}

template <bool kF8>
__device__ void produce(const Params& p, Ctrl* ctrl, uint8_t* ring, const CUtensorMap* tm_s, const CUtensorMap* tm_pe,
                        const CUtensorMap* tm_qn, const CUtensorMap* tm_qp) {
  using C = chunk::Cfg<kF8, 1>;
  volatile int* abort = &ctrl->abort;
  UnitIter it;
  it.init(p, ctrl);
  Unit u;
  uint32_t i = 0, un = 0, qloaded = 0;
  bool ok = true;
  auto acquire = [&]() -> bool {
    const int st = static_cast<int>(i % C::kNStS);
    return mbar_wait(smem_u32(&ctrl->kv_empty[st]), ((i / C::kNStS) & 1) ^ 1, abort, p.timeout_ns);
  };
  while (ok && it.next(u)) {
    const uint32_t qbar = smem_u32(&ctrl->q_bar[un & 1]);
    for (int e = 0; e < C::kQEntries; ++e, ++i) {
      if (!acquire()) {
        ok = false;
        break;
      }
      const int st = static_cast<int>(i % C::kNStS);
      if (e == 0) {
        mbar_expect_tx(qbar, static_cast<uint32_t>(kRows * 1152));
        qloaded = un + 1;
      }
      mbar_arrive(smem_u32(&ctrl->kv_full[st]));
      const int row = u.b * p.R + C::kQRows * e;
      const uint32_t slot = smem_u32(ring + st * C::kSlotS);
      tma_load_3d(slot, tm_qn, 0, row, 0, qbar);
      tma_load_2d(slot + C::kQRows * 128 * 8, tm_qp, 0, row, qbar);
    }
    ++un;
    for (int pg = u.p0; pg < u.p1 && ok; ++pg) {
      int32_t pid = __ldg(p.page_table + static_cast<int64_t>(u.b) * p.pt_stride + pg);
      if (pid < 0 || pid >= p.num_pages) {
        atomicOr(p.status, MLA_DEV_BAD_PAGE_ID);
        pid = 0;
      }
      if (!acquire()) {
        ok = false;
        break;
      }
      const int st = static_cast<int>(i % C::kNStS);
      const uint32_t bar = smem_u32(&ctrl->kv_full[st]), slot = smem_u32(ring + st * C::kSlotS);
      mbar_expect_tx(bar, static_cast<uint32_t>(C::kSlotS));
      tma_load_3d(slot, tm_s, 0, pid * kPage, 0, bar);
      if constexpr (kF8) tma_load_2d(slot + C::kSBoxes * C::kBox, tm_pe, kDL, pid * kPage, bar);
      ++i;
    }
  }
  if (!ok) raise_timeout(p, ctrl, kWaitEmpty, i);
  for (uint32_t q = 0; q < static_cast<uint32_t>(C::kNStS) && q < i; ++q) {  // every copy has landed before exit
    const uint32_t last = i - 1 - ((i - 1 - q) % C::kNStS);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(&ctrl->kv_full[q]), (last / C::kNStS) & 1) && globaltimer_ns() - t0 < p.timeout_ns) {
    }
  }
  if (qloaded) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(&ctrl->q_bar[(qloaded - 1) & 1]), ((qloaded - 1) >> 1) & 1) &&
           globaltimer_ns() - t0 < p.timeout_ns) {
    }
  }
}

template <bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
    mla_mass_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_s,
                    const __grid_constant__ CUtensorMap tm_pe, const __grid_constant__ CUtensorMap tm_qn,
                    const __grid_constant__ CUtensorMap tm_qp) {
  using C = chunk::Cfg<kF8, 1>;
  using M = Lay<kF8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* data = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(data + M::kData);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < chunk::kMaxStages; ++i) {
      mbar_init(smem_u32(&ctrl->kv_full[i]), 1);
      mbar_init(smem_u32(&ctrl->kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctrl->q_bar[i]), 1);
      mbar_init(smem_u32(&ctrl->sums[i]), 4);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(smem_u32(&ctrl->s_full[i]), 1);
      mbar_init(smem_u32(&ctrl->s_empty[i]), 4);
    }
    mbar_init(smem_u32(&ctrl->q_full), 8);
    mbar_init(smem_u32(&ctrl->drain), 1);
    ctrl->abort = 0;
    ctrl->first = p.B;
    ctrl->start = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_s);
    tma_prefetch_desc(&tm_qn);
    tma_prefetch_desc(&tm_qp);
    if (kF8) tma_prefetch_desc(&tm_pe);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&ctrl->tmem_base), 512);
    tmem_relinquish();
  }
  // A request occupies kUnitCost + pages of the weighted line.
  const bool bad = find_slice(p, ctrl, [&](int L) { return kUnitCost + (L + kPage - 1) / kPage; });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the status words are cleared
  griddep_launch_dependents();
  if (bad && blockIdx.x == 0) atomicOr(p.status, MLA_DEV_BAD_SEQ_LEN);
  const uint32_t tmem = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;
  uint8_t* ring = data;

  if (warp == 0) {
    if (lane == 0) produce<kF8>(p, ctrl, ring, &tm_s, &tm_pe, &tm_qn, &tm_qp);
  } else if (warp == 1) {
    UnitIter it;
    it.init(p, ctrl);
    Unit u;
    uint32_t i = 0, j = 0, un = 0;
    bool ok = true;
    int why = 0;
    while (ok && it.next(u)) {
      for (int e = 0; e < C::kQEntries && ok; ++e, ++i)  // no phase of an entry is ever skipped
        ok = mbar_wait_warp(smem_u32(&ctrl->kv_full[i % C::kNStS]), (i / C::kNStS) & 1, abort, p.timeout_ns);
      why = kWaitLanded;
      if (!ok) break;
      if (!mbar_wait_warp(smem_u32(&ctrl->q_full), un & 1, abort, p.timeout_ns)) {
        ok = false;
        why = kWaitQFull;
        break;
      }
      if (lane == 0)
        for (int e = C::kQEntries; e > 0; --e) mbar_arrive(smem_u32(&ctrl->kv_empty[(i - e) % C::kNStS]));
      __syncwarp();
      ++un;
      for (int pg = u.p0; pg < u.p1; ++pg, ++j, ++i) {
        const int st = static_cast<int>(i % C::kNStS), sb = static_cast<int>(j % 3);
        if (!mbar_wait_all_warp(smem_u32(&ctrl->kv_full[st]), (i / C::kNStS) & 1, smem_u32(&ctrl->s_empty[sb]),
                                ((j / 3) & 1) ^ 1, 0u, 0u, 0u, 0u, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitLanded;
          break;
        }
        tc_fence_after();
        const uint32_t slot = smem_u32(ring + st * C::kSlotS);
        const uint64_t dlat = smem_desc(slot, 16, 1024, kSwizzle128B);
        const uint32_t dcol = tmem + C::kSCol0 + sb * 64;
        if constexpr (!kF8) {
#pragma unroll
          for (int d = 0; d < 9; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts_e<false>(dcol, tmem + d * 32 + k * 8, dlat + static_cast<uint64_t>(d * (C::kBox >> 4) + k * 2),
                              C::kIdescQK, (d | k) ? 1u : 0u);
        } else {
          const uint64_t dpe = smem_desc(slot + C::kSBoxes * C::kBox, 16, 512, kSwizzle64B);
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const uint32_t qcol = tmem + (term ? C::kQLoCol : 0u);
#pragma unroll
            for (int d = 0; d < 4; ++d)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts_e<true>(dcol, qcol + d * 32 + k * 8, dlat + static_cast<uint64_t>(d * (C::kBox >> 4) + k * 2),
                               C::kIdescQK, (term | d | k) ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma_ts_e<true>(dcol, qcol + 128 + k * 8, dpe + static_cast<uint64_t>(k * 2), C::kIdescQK, 1u);
          }
        }
        mma_commit_e(smem_u32(&ctrl->kv_empty[st]));
        mma_commit_e(smem_u32(&ctrl->s_full[sb]));
      }
    }
    if (!ok && lane == 0) raise_timeout(p, ctrl, why, j);
    __syncwarp();
    mma_commit_e(smem_u32(&ctrl->drain));
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&ctrl->drain), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int r = (warp & 3) * 32 + lane;
    const int gg = (warp - 4) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* sums = reinterpret_cast<float*>(data + M::kSums) + gg * 2 * 4 * 64;
    UnitIter it;
    it.init(p, ctrl);
    Unit u;
    uint32_t i = 0, j = 0, un = 0, n = 0;  // n: pages of this group
    bool ok = true;
    int why = 0;
    while (ok && it.next(u)) {
      if (j > 0 && !mbar_wait_warp<false, true>(smem_u32(&ctrl->s_full[(j - 1) % 3]), ((j - 1) / 3) & 1, abort,
                                                p.timeout_ns)) {
        ok = false;
        why = kWaitSPrev;
        break;
      }
      if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->q_bar[un & 1]), (un >> 1) & 1, abort, p.timeout_ns)) {
        ok = false;
        why = kWaitQ;
        break;
      }
      const int row = r;  // of the request's R <= 128 rows
      const bool real = row < p.R;
      float nl = 0.f;  // -lse in log2 units
      int nvis = 0;
      if (real) {
        const float l = p.lse[static_cast<int64_t>(u.b) * p.R + row];
        nvis = l == -INFINITY ? 0 : u.L - p.Q + row / p.H + 1;
        nl = -l * kLog2e;
      }
      float qs = 1.f;
      if constexpr (kF8) {
        qs = chunk::q_row_scale<1>(ring, i, r);
        chunk::q_row_e4m3<1>(ring, i, r, tmem + lane_base, nullptr, gg == 0 ? 0 : 5, gg == 0 ? 5 : 9, qs);
      } else {
        chunk::q_row_bf16<1, 36>(ring, i, r, tmem + lane_base, 36 * gg);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl->q_full));
      i += C::kQEntries + static_cast<uint32_t>(u.p1 - u.p0);
      ++un;
      const float c2 = kF8 ? p.c2 * qs : p.c2;  // qs is a power of two
      const float* in = p.mass_in ? p.mass_in + static_cast<int64_t>(u.b) * p.cols : nullptr;
      float* out = p.mass_out + static_cast<int64_t>(u.b) * p.cols;
      const int old = u.L - p.num_fresh;  // tokens below start from mass_in
      for (int pg = u.p0; pg < u.p1; ++pg, ++j) {
        if ((pg & 1) != gg) continue;
        const int sb = static_cast<int>(j % 3);
        const int t0 = pg * kPage, t = t0 + r;
        float base = 0.f;
        if (r < 64 && t < old && in) base = in[t];
        if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->s_full[sb]), (j / 3) & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitS;
          break;
        }
        tc_fence_after();
        uint32_t v[4][16];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld16(tmem + lane_base + C::kSCol0 + sb * 64 + q * 16, v[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_wait_ld_tie(v[q]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->s_empty[sb]));
        float f[64];
        const int z = nvis - t0;  // keys of the page that the row sees
        if (__all_sync(0xffffffffu, z >= kPage)) {
#pragma unroll
          for (int k = 0; k < 64; ++k) f[k] = ex2_approx(fmaf(__uint_as_float(v[k >> 4][k & 15]), c2, nl));
        } else {  // unseen keys, padding rows: exactly 0, whatever the slot holds
#pragma unroll
          for (int k = 0; k < 64; ++k) {
            const float e = ex2_approx(fmaf(__uint_as_float(v[k >> 4][k & 15]), c2, nl));
            f[k] = k < z ? e : 0.f;
          }
        }
        // halving exchanges: lane l ends with the warp's sums of keys 2 l, 2 l + 1
#pragma unroll
        for (int o = 16, w = 32; w >= 2; o >>= 1, w >>= 1) {
          const bool hi = (lane & o) != 0;
#pragma unroll
          for (int k = 0; k < w; ++k) {
            const float keep = hi ? f[k + w] : f[k], send = hi ? f[k] : f[k + w];
            f[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
        float* s4 = sums + (n & 1) * 256;
        *reinterpret_cast<float2*>(s4 + (warp & 3) * 64 + 2 * lane) = make_float2(f[0], f[1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->sums[gg]));
        // all four warps wait, so that none gets two pages ahead of another
        if (!mbar_wait_warp(smem_u32(&ctrl->sums[gg]), n & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitSums;
          break;
        }
        ++n;
        if (r < 64 && t < u.L) out[t] = base + ((s4[r] + s4[64 + r]) + (s4[128 + r] + s4[192 + r]));
      }
    }
    if (!ok && lane == 0) raise_timeout(p, ctrl, why, j);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
}

// ------------------------------------------- many rows: the keys stay
constexpr int kKeys = 128;   // keys of a tile (M of the MMAs)
constexpr int kSlot = 73728;  // a page of the cache, or 64 query rows
constexpr int kSlots = 3;
constexpr int kFull = 2 * kSlots;  // barriers of the ring's entries: two rounds, see the issuing warps
// Barriers that say a row tile is scored (tile j: barrier j % 6, phase j / 6),
// two rounds of the three score buffers.  A parity wait for a phase also passes
// while the phase two before it was the last to complete, so whoever waits for
// tile j must know that tile j - 6 is complete, and tile j + 6 must not
// complete before the wait has passed.  A row group knows of j - 6: it has the
// same parity, so the group read it itself.  And j + 6 needs j + 3 read out of
// the score buffer, which was not issued before this group had read j.  (With
// three barriers a group would have to know of tile j - 3, which the other
// group reads and the other warp issues: where its rows land late, tile j - 2
// comes first and the wait for j passes at once.)
constexpr int kScoreFull = 6;
constexpr int kNlOff = kSlots * kSlot;            // [3][64] -lse of a row tile, in log2 units
constexpr int kPartOff = kNlOff + 3 * 64 * 4;     // [2][128] the second group's sums
constexpr int kClusOff = kPartOff + 2 * kKeys * 4;  // [8][128] the sums of the cluster's CTAs (in its first)
constexpr int kRowsData = kClusOff + 8 * kKeys * 4;
constexpr int kRowsSmem = 1024 + kRowsData + 512;

// The key tiles of a CTA's slice, in order.
struct Tile {
  int b, L, t0;  // keys t0 .. t0 + 127
};
struct TileIter {
  const Params* p;
  long long x, x1, start;
  int b;
  __device__ void init(const Params& pp, const Ctrl* c) {
    p = &pp;
    const int n = gridDim.x / pp.cluster, i = blockIdx.x / pp.cluster;
    x = c->total * i / n;
    x1 = c->total * (i + 1) / n;
    start = c->start;
    b = c->first;
  }
  __device__ bool next(Tile& u) {
    while (x < x1 && b < p->B) {
      u.L = length_of(*p, b);
      const long long tiles = (u.L + kKeys - 1) / kKeys;
      if (x >= start + tiles) {
        start += tiles;
        ++b;
        continue;
      }
      u.b = b;
      u.t0 = static_cast<int>(x - start) * kKeys;
      ++x;
      return true;
    }
    return false;
  }
};

// 16 codes (a 16-byte chunk) as 16 bf16 values (exact).
__device__ __forceinline__ void expand16(uint4 v, uint32_t* o) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(in[k] >> (16 * h)), __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
      const __nv_bfloat162 b2 = __floats2bfloat162_rn(f.x, f.y);
      o[2 * k + h] = *reinterpret_cast<const uint32_t*>(&b2);
    }
}

template <bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
    mla_mass_rows_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_s,
                         const __grid_constant__ CUtensorMap tm_pe, const __grid_constant__ CUtensorMap tm_qn,
                         const __grid_constant__ CUtensorMap tm_qp) {
  using C = chunk::Cfg<false, 1>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* data = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(data + kRowsData);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kFull; ++i) mbar_init(smem_u32(&ctrl->kv_full[i]), 1);
    for (int i = 0; i < kScoreFull; ++i) mbar_init(smem_u32(&ctrl->s_full[i]), 2);  // a tile's QK, its -lse (warp 3)
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&ctrl->s_empty[i]), 4);          // the group that read it
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ctrl->q_bar[i]), 1);
      mbar_init(smem_u32(&ctrl->sums[i]), 4);
    }
    mbar_init(smem_u32(&ctrl->q_full), 8);
    mbar_init(smem_u32(&ctrl->drain), 2);  // both issuing warps
    ctrl->abort = 0;
    ctrl->first = p.B;
    ctrl->start = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_s);
    tma_prefetch_desc(&tm_qn);
    tma_prefetch_desc(&tm_qp);
    if (kF8) tma_prefetch_desc(&tm_pe);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&ctrl->tmem_base), 512);
    tmem_relinquish();
  }
  const bool bad = find_slice(p, ctrl, [&](int L) { return (L + kKeys - 1) / kKeys; });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (p.cluster > 1) {  // the first CTA has begun before the others write to its shared memory
    __syncwarp();
    cluster_sync();
  }
  griddep_wait();
  griddep_launch_dependents();
  if (bad && blockIdx.x == 0) atomicOr(p.status, MLA_DEV_BAD_SEQ_LEN);
  const uint32_t tmem = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;
  uint8_t* ring = data;
  // row tiles first, first + step .. of the request are this CTA's
  const int all_tiles = (p.R + 63) / 64, step = p.cluster, first = static_cast<int>(blockIdx.x) % p.cluster;
  TileIter it;
  it.init(p, ctrl);
  Tile u;
  uint32_t un = 0;
  bool ok = true;
  int why = 0;

  if (warp == 0) {
    if (lane == 0) {
      // per key tile its pages (ring entries that complete on q_bar), then
      // the request's row tiles.  An entry's slot is free once the rows that
      // it held are scored (s_full) or the keys are in TMEM (q_full): no
      // commit of their own (a commit and its wait cost the issuing warp
      // about as long as four MMAs).
      uint32_t i = 0, j = 0;
      uint32_t held[kSlots] = {0, 0, 0};  // entries i - 3, i - 2, i - 1: 2 tile, or 2 unit + 1
      auto acquire = [&](uint32_t what) -> bool {
        if (i >= kSlots) {
          const uint32_t k = held[0] >> 1;
          if (!mbar_wait(smem_u32(held[0] & 1u ? &ctrl->q_full : &ctrl->s_full[k % kScoreFull]),
                         (held[0] & 1u ? k : k / kScoreFull) & 1, abort, p.timeout_ns))
            return false;
        }
        held[0] = held[1];
        held[1] = held[2];
        held[2] = what;
        return true;
      };
      while (ok && it.next(u)) {
        const uint32_t qbar = smem_u32(&ctrl->q_bar[un & 1]);
        const int pages = u.t0 + kPage < u.L ? 2 : 1;
        for (int e = 0; e < 2; ++e, ++i) {
          if (!acquire(2 * un + 1)) {
            ok = false;
            break;
          }
          const uint32_t slot = smem_u32(ring + (i % kSlots) * kSlot);
          if (e == 0) mbar_expect_tx(qbar, static_cast<uint32_t>(pages * kPage * (kF8 ? 576 : 1152)));
          mbar_arrive(smem_u32(&ctrl->kv_full[i % kFull]));
          if (e >= pages) continue;  // an odd last page: its lanes are not stored
          int32_t pid = __ldg(p.page_table + static_cast<int64_t>(u.b) * p.pt_stride + u.t0 / kPage + e);
          if (pid < 0 || pid >= p.num_pages) {
            atomicOr(p.status, MLA_DEV_BAD_PAGE_ID);
            pid = 0;
          }
          tma_load_3d(slot, &tm_s, 0, pid * kPage, 0, qbar);
          if constexpr (kF8) tma_load_2d(slot + 4 * 8192, &tm_pe, kDL, pid * kPage, qbar);
        }
        ++un;
        for (int n = first; n < all_tiles && ok; n += step, ++i, ++j) {
          if (!acquire(2 * j)) {
            ok = false;
            break;
          }
          const uint32_t slot = smem_u32(ring + (i % kSlots) * kSlot), bar = smem_u32(&ctrl->kv_full[i % kFull]);
          const int row = u.b * p.R + 64 * n;
          mbar_expect_tx(bar, static_cast<uint32_t>(kSlot));
          tma_load_3d(slot, &tm_qn, 0, row, 0, bar);
          tma_load_2d(slot + 8 * 8192, &tm_qp, 0, row, bar);
        }
      }
      if (!ok) raise_timeout(p, ctrl, kWaitEmpty, i);
      for (uint32_t q = 0; q < static_cast<uint32_t>(kFull) && q < i; ++q) {
        const uint32_t last = i - 1 - ((i - 1 - q) % kFull);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&ctrl->kv_full[q]), (last / kFull) & 1) && globaltimer_ns() - t0 < p.timeout_ns) {
        }
      }
      if (un) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&ctrl->q_bar[(un - 1) & 1]), ((un - 1) >> 1) & 1) &&
               globaltimer_ns() - t0 < p.timeout_ns) {
        }
      }
    }
  } else if (warp < 3) {
    // Warps 1 and 2 issue the even and the odd row tiles: what a warp spends on
    // a wait and a commit (~230 cycles beside the row warps) passes while the
    // other one's MMAs run.  A warp waits for its own tiles alone.  No phase
    // can pass it by: an entry's barrier comes again six entries later, when
    // the slot has been used once more, and that needs this entry consumed.
    // (Every key tile has row tiles of both warps, or is the CTA's only one.)
    uint32_t i = 0, j = 0;
    while (ok && it.next(u)) {
      i += 2;
      if (!mbar_wait_warp(smem_u32(&ctrl->q_full), un & 1, abort, p.timeout_ns)) {
        ok = false;
        why = kWaitQFull;
        break;
      }
      ++un;
      for (int n = first; n < all_tiles; n += step, ++j, ++i) {
        if ((j & 1u) != static_cast<uint32_t>(warp - 1)) continue;
        const int st = static_cast<int>(i % kSlots), sb = static_cast<int>(j % 3);
        // (that this tile has landed also says that the tile three before it,
        // whose score buffer it takes, was issued)
        if (!mbar_wait_all_warp(smem_u32(&ctrl->kv_full[i % kFull]), (i / kFull) & 1, smem_u32(&ctrl->s_empty[sb]),
                                ((j / 3) & 1) ^ 1, 0u, 0u, 0u, 0u, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitLanded;
          break;
        }
        tc_fence_after();
        const uint64_t dq = smem_desc(smem_u32(ring + st * kSlot), 16, 1024, kSwizzle128B);
        const uint32_t dcol = tmem + C::kSCol0 + sb * 64;
#pragma unroll
        for (int d = 0; d < 9; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts_e<false>(dcol, tmem + d * 32 + k * 8, dq + static_cast<uint64_t>(d * (8192 >> 4) + k * 2),
                            C::kIdescQK, (d | k) ? 1u : 0u);
        mma_commit_e(smem_u32(&ctrl->s_full[j % kScoreFull]));
      }
    }
    if (!ok && lane == 0) raise_timeout(p, ctrl, why, j);
    __syncwarp();
    mma_commit_e(smem_u32(&ctrl->drain));
    if (lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&ctrl->drain), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // -lse of every row tile, in log2 units, beside the score buffer it
    // belongs to; -inf (a weight of 0) for rows that saw nothing
    uint32_t j = 0;
    float* nl = reinterpret_cast<float*>(data + kNlOff);
    while (ok && it.next(u)) {
      const float* lse = p.lse + static_cast<int64_t>(u.b) * p.R;
      for (int n = first; n < all_tiles; n += step, ++j) {
        const int sb = static_cast<int>(j % 3);
        float v[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int row = 64 * n + lane + 32 * q;
          const float l = row < p.R ? lse[row] : INFINITY;
          v[q] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        }
        if (!mbar_wait_warp(smem_u32(&ctrl->s_empty[sb]), ((j / 3) & 1) ^ 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitOther;
          break;
        }
        nl[sb * 64 + lane] = v[0];
        nl[sb * 64 + 32 + lane] = v[1];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->s_full[j % kScoreFull]));
      }
    }
    if (!ok && lane == 0) raise_timeout(p, ctrl, why, j);
  } else if (warp >= 4) {
    const int r = (warp & 3) * 32 + lane;  // key of the tile
    const int gg = (warp - 4) >> 2;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float c2 = p.c2;
    float* parts = reinterpret_cast<float*>(data + kPartOff);
    uint32_t i = 0, j = 0;
    while (ok && it.next(u)) {
      // the tile's keys replace the earlier ones in TMEM once every QK with
      // those is done: the last tile of either issuing warp
      for (uint32_t back = 1; back <= 2 && ok; ++back)
        ok = j < back || mbar_wait_warp<false, true>(smem_u32(&ctrl->s_full[(j - back) % kScoreFull]),
                                                     ((j - back) / kScoreFull) & 1, abort, p.timeout_ns);
      if (!ok) {
        why = kWaitSPrev;
        break;
      }
      if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->q_bar[un & 1]), (un >> 1) & 1, abort, p.timeout_ns)) {
        ok = false;
        why = kWaitQ;
        break;
      }
      const uint8_t* src = ring + ((i + (r >> 6)) % kSlots) * kSlot;
      const int row = r & 63;
      if constexpr (kF8) {
        // chunks of 16 codes: 32 of c_kv in four 128-byte columns, 4 of k_pe
        // in 64-byte rows; group gg takes pairs [9 gg, 9 gg + 9)
#pragma unroll 3
        for (int q = 9 * gg; q < 9 * gg + 9; ++q) {
          uint32_t w[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 2 * q + h;
            const uint8_t* a = c < 32 ? src + (c >> 3) * 8192 + row * 128 + (((c & 7) ^ (row & 7)) << 4)
                                      : src + 4 * 8192 + row * 64 + (((c - 32) ^ ((row >> 1) & 3)) << 4);
            expand16(*reinterpret_cast<const uint4*>(a), w + 8 * h);
          }
          tmem_st16(tmem + lane_base + 16 * q, w);
        }
      } else {
#pragma unroll 3
        for (int q = 9 * gg; q < 9 * gg + 9; ++q) {  // four chunks of 8 values
          uint32_t w[16];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int c = 4 * q + h;
            const uint4 v = *reinterpret_cast<const uint4*>(src + (c >> 3) * 8192 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
            w[4 * h] = v.x; w[4 * h + 1] = v.y; w[4 * h + 2] = v.z; w[4 * h + 3] = v.w;
          }
          tmem_st16(tmem + lane_base + 16 * q, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctrl->q_full));
      i += 2 + (all_tiles - first + step - 1) / step;
      const int t = u.t0 + r;
      // the first row that sees the key: rows of the positions from t on
      const int64_t first_pos = static_cast<int64_t>(t) - (u.L - p.Q);
      const int64_t rmin = t < u.L ? (first_pos > 0 ? first_pos * p.H : 0) : p.R;
      float sum4[4] = {0.f, 0.f, 0.f, 0.f};
      for (int n = first; n < all_tiles; n += step, ++j) {
        if ((j & 1u) != static_cast<uint32_t>(gg)) continue;
        const int sb = static_cast<int>(j % 3);
        if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->s_full[j % kScoreFull]), (j / kScoreFull) & 1, abort,
                                         p.timeout_ns)) {
          ok = false;
          why = kWaitS;
          break;
        }
        tc_fence_after();
        uint32_t v[4][16];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld16(tmem + lane_base + C::kSCol0 + sb * 64 + q * 16, v[q]);
        float4 l[16];
        const float4* nl = reinterpret_cast<const float4*>(data + kNlOff + sb * 256);
#pragma unroll
        for (int q = 0; q < 16; ++q) l[q] = nl[q];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_wait_ld_tie(v[q]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->s_empty[sb]));
        // columns [a, z) of the tile count: from the first row that sees the
        // key to the request's last row
        const int64_t a64 = rmin - 64 * n;
        const int a = a64 > 0 ? (a64 < 64 ? static_cast<int>(a64) : 64) : 0;
        const int z = p.R - 64 * n < 64 ? p.R - 64 * n : 64;
        if (__all_sync(0xffffffffu, a == 0) && z == 64) {
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            sum4[0] += ex2_approx(fmaf(__uint_as_float(v[q >> 2][(4 * q) & 15]), c2, l[q].x));
            sum4[1] += ex2_approx(fmaf(__uint_as_float(v[q >> 2][(4 * q + 1) & 15]), c2, l[q].y));
            sum4[2] += ex2_approx(fmaf(__uint_as_float(v[q >> 2][(4 * q + 2) & 15]), c2, l[q].z));
            sum4[3] += ex2_approx(fmaf(__uint_as_float(v[q >> 2][(4 * q + 3) & 15]), c2, l[q].w));
          }
        } else {
          const float* lf = reinterpret_cast<const float*>(l);
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            const float e = ex2_approx(fmaf(__uint_as_float(v[c >> 4][c & 15]), c2, lf[c]));
            sum4[c & 3] += (c >= a && c < z) ? e : 0.f;
          }
        }
      }
      if (!ok) break;
      const float sum = (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
      // the second group hands its sums over; it writes the next ones into
      // this buffer two tiles later, whose keys need the first group's q_full
      float* part = parts + (un & 1) * kKeys;
      if (gg == 1) {
        part[r] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->sums[un & 1]));
      } else {
        if (!mbar_wait_warp(smem_u32(&ctrl->sums[un & 1]), (un >> 1) & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitSums;
          break;
        }
        if (step > 1) {  // added up below
          st_cluster_u32(mapa(smem_u32(data + kClusOff) + (first * kKeys + r) * 4, 0), __float_as_uint(sum + part[r]));
        } else if (t < u.L) {
          const int64_t at = static_cast<int64_t>(u.b) * p.cols + t;
          const float base = p.mass_in && t < u.L - p.num_fresh ? p.mass_in[at] : 0.f;
          p.mass_out[at] = base + (sum + part[r]);
        }
      }
      ++un;
    }
    if (!ok && lane == 0) raise_timeout(p, ctrl, why, j);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, 512);
  if (step > 1) {  // a cluster has one key tile at most (cluster_of)
    __syncwarp();
    cluster_sync();
    TileIter last;
    last.init(p, ctrl);
    const int r = tid;
    if (first == 0 && r < kKeys && last.next(u) && u.t0 + r < u.L && !*abort) {
      const int t = u.t0 + r;
      const int64_t at = static_cast<int64_t>(u.b) * p.cols + t;
      float sum = p.mass_in && t < u.L - p.num_fresh ? p.mass_in[at] : 0.f;
      const float* parts = reinterpret_cast<const float*>(data + kClusOff);
      float add = 0.f;
      for (int q = 0; q < step; ++q) add += parts[q * kKeys + r];
      p.mass_out[at] = sum + add;
    }
  }
}

}  // namespace mass
}  // namespace mla

namespace {

using mla::chunk::Cfg;
using mla::mass::Lay;
using mla::mass::Params;
using namespace mla::host;

int check_mass_dims(const mla_dims* d) {
  if (!d || d->batch < 1 || d->num_heads < 1 || d->q_len < 1 || d->num_pages < 1 || d->max_pages_per_req < 1 ||
      d->page_table_stride < d->max_pages_per_req)
    return MLA_ERR_INVALID_ARG;
  if (d->page_size != 64) return MLA_ERR_UNSUPPORTED;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  const int64_t B = d->batch;
  if (static_cast<int64_t>(d->num_pages) * 64 > INT_MAX || B * d->max_pages_per_req > (1 << 30) / 64 ||
      B * d->q_len > INT_MAX || B * d->q_len * d->num_heads > INT_MAX)
    return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

template <int kTag, typename Kernel>
cudaError_t launch_mass(Kernel* kernel, int smem, const Params& p, const CUtensorMap& s, const CUtensorMap& pe,
                        const CUtensorMap& qn, const CUtensorMap& qp, int ctas, unsigned cluster, int device,
                        cudaStream_t stream) {
  cudaError_t e = allow_smem<kTag>(kernel, smem, device);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(ctas), dim3(mla::chunk::kThreads), smem, stream, cluster, p, s, pe, qn, qp);
}

}  // namespace

extern "C" {

size_t mla_attn_mass_workspace_size(const mla_dims* d, int device) {
  (void)device;
  return check_mass_dims(d) == MLA_OK ? 256 : 0;
}

int mla_attn_mass(const mla_dims* d, const void* q_nope, const void* q_pe, const void* kv_cache,
                  const int32_t* page_table, const int32_t* seq_lens, const float* lse, int32_t num_fresh, float scale,
                  float kv_scale, const float* mass, float* mass_out, int32_t mass_cols, void* workspace,
                  size_t workspace_bytes, void* stream_v) {
  int rc = check_mass_dims(d);
  if (rc != MLA_OK) return rc;
  if (!q_nope || !q_pe || !kv_cache || !page_table || !seq_lens || !lse || !mass_out || !workspace || mass_cols < 1 ||
      num_fresh < 0)
    return MLA_ERR_INVALID_ARG;
  const bool f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  if (!scale_ok(scale, kv_scale, f8)) return MLA_ERR_INVALID_ARG;
  if (!aligned(q_nope, 32) || !aligned(q_pe, 32) || !aligned(kv_cache, 16) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(mass, 4) || !aligned(mass_out, 4) || !aligned(workspace, 256))
    return MLA_ERR_ALIGNMENT;
  if (workspace_bytes < 256) return MLA_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  if ((rc = device_ok(dev)) != MLA_OK) return rc;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return MLA_ERR_CUDA;
  if (!encode_fn() || !mla::host::bind_context(dev)) return MLA_ERR_CUDA;
  const int64_t R = static_cast<int64_t>(d->num_heads) * d->q_len;
  const int64_t krows = static_cast<int64_t>(d->num_pages) * 64, qrows = d->batch * R;
  // more than 128 rows per request: the keys stay and the rows stream (64 at
  // a time)
  const bool rows = R > mla::chunk::kRows;
  CUtensorMap s, pe, qn, qp;
  bool ok = true;
  if (f8) {
    using C = Cfg<true, 1>;
    ok = map3(&s, kv_cache, krows, 576, 1, C::kSBoxes, 64, C::kPartBoxes) &&
         map2(&pe, kv_cache, krows, 576, 1, 64, 64, CU_TENSOR_MAP_SWIZZLE_64B) &&
         map3(&qn, q_nope, qrows, 1024, 2, 8, rows ? 64 : C::kQRows, 8) &&
         map2(&qp, q_pe, qrows, 64, 2, 64, rows ? 64 : C::kQRows, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    using C = Cfg<false, 1>;
    ok = map3(&s, kv_cache, krows, 1152, 2, C::kSBoxes, 64, C::kPartBoxes) &&
         map3(&qn, q_nope, qrows, 1024, 2, 8, rows ? 64 : C::kQRows, 8) &&
         map2(&qp, q_pe, qrows, 64, 2, 64, rows ? 64 : C::kQRows, CU_TENSOR_MAP_SWIZZLE_128B);
    pe = s;
  }
  if (!ok) return MLA_ERR_CUDA;
  Params p;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.lse = lse;
  p.mass_in = mass;
  p.mass_out = mass_out;
  p.status = static_cast<int32_t*>(workspace);
  p.B = d->batch;
  p.H = d->num_heads;
  p.Q = d->q_len;
  p.R = static_cast<int32_t>(R);
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages_per_req;
  p.pt_stride = d->page_table_stride;
  p.cols = mass_cols;
  p.cap = d->max_pages_per_req * 64 < mass_cols ? d->max_pages_per_req * 64 : mass_cols;
  p.num_fresh = num_fresh;
  // CTAs per key tile, by the most tiles that the lengths allow
  p.cluster = rows ? mla::mass::cluster_of(
                         static_cast<int64_t>(d->batch) * ((p.cap + mla::mass::kKeys - 1) / mla::mass::kKeys), R, sms)
                   : 1;
  p.c2 = log2_scale(scale, f8 ? kv_scale : 1.f);
  p.timeout_ns = 2000000000ull;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  cudaError_t e = launch_pdl(mla::mass::mla_mass_clear_kernel, dim3(1), dim3(32), 0, stream, 0, p.status);
  if (e == cudaSuccess) {
    using namespace mla::mass;
    const unsigned cl = p.cluster > 1 ? p.cluster : 0;
    const int ctas = sms / p.cluster * p.cluster;
    e = rows ? (f8 ? launch_mass<3>(mla_mass_rows_kernel<true>, kRowsSmem, p, s, pe, qn, qp, ctas, cl, dev, stream)
                   : launch_mass<2>(mla_mass_rows_kernel<false>, kRowsSmem, p, s, pe, qn, qp, ctas, cl, dev, stream))
             : (f8 ? launch_mass<1>(mla_mass_kernel<true>, Lay<true>::kSmem, p, s, pe, qn, qp, ctas, cl, dev, stream)
                   : launch_mass<0>(mla_mass_kernel<false>, Lay<false>::kSmem, p, s, pe, qn, qp, ctas, cl, dev, stream));
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // extern "C"

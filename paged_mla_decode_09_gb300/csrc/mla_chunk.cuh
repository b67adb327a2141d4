// Device code of the chunk attention behind mla_prefill and
// mla_decode_window: schedule, split-KV attention, log-sum-exp combine.
//
// Row r of the flattened queries [T * H] belongs to token r / H, head r % H.
// A request's rows are cut into blocks of kCg * 128 consecutive rows; a
// block's keys are the pages that any of its rows sees: with a window the
// sink pages, then the window's pages (a virtual page index v maps to the
// real page v, or v + skip behind the sink pages).  Over those pages each
// row computes, with one pass and a running maximum,
//
//     s_t = (q_nope . c_kv[t] + q_pe . k_pe[t]) * scale,  P = 2^(s log2e - R),
//     O = sum P c_kv[t],  l = sum P,  out = O / l,  lse = (R + log2 l) ln 2.
//
// What bounds it: 2176 flops per (row, key) on the tensor pipe once a block
// is full, the cache's bytes from HBM when a request has few rows.  How it is
// laid out: an O accumulator of 128 rows x 512 fp32 fills an SM's tensor
// memory, so scores and outputs live in different SMs.
//   * S CTA: the block's queries in TMEM (A operand), pages K-major in shared
//     memory (B), S = Q K^T of 64 keys at a time, softmax (one thread per
//     row), P sent to its O CTA by st.async;
//   * O CTA: O += P V, V = the same page through an MN-major descriptor.
// kCg = 1: one S/O pair (cluster of 2) per 128 rows.  kCg = 2: two S CTAs and
// two O CTAs (cluster of 4) per 256 rows, each pair running cta_group::2
// MMAs of M = 256.  A pair's CTAs hold half of B each, so every SM copies in
// and reads half the page bytes per MMA: at M = 128 the S CTA's page copies
// and operand reads (72 KB each per 1152 tensor cycles) alone take the 128
// bytes a cycle that shared memory has.  A pair scores 128 keys at a time
// (one page in each S CTA): an MMA of N = 64 lasts 32 cycles, no longer than
// its issue takes, so that every wait of the issuing warp (~200 cycles each)
// left the tensor pipe idle; at N = 128 the queue covers one wait per tile.
// Measured: 2 x 512 tokens x 128 heads over 8K keys 1279 us (1885 TFLOP/s;
// 1738 in a loop, under the power limit), the tensor pipes 87.6 % busy.
//
// An e4m3 cache: QK runs on the codes as they are (kind::f8f6f4), the queries
// as two e4m3 terms hi + lo of q / 2^k.  A bf16 value has 8 significant bits
// and hi + lo hold 4 + 4, so with a power-of-two row scale the split is exact
// down to 2^-10 of the row's largest value and scores are as exact as with a
// bf16 cache.  PV runs in f16: the O CTA's row warps expand the codes
// (exact in f16) into the V ring, and P keeps f16's range (P as e4m3 terms
// loses the many small weights of a long row to subnormals).  f16 weights end
// 2^-25 below the reference, which is at most the row's maximum: beside a token
// that scores 20 above all others the others of its piece are lost to out, which
// shows if that token's values are near 0 (one such token of 2000, in pieces:
// 0.3 % of the output at 14, 6 % at 17, 15 % from 20 on).  bf16 weights on codes expanded to bf16 would keep
// them, at 3 bits less in every weight: ordinary inputs' outputs would be 0.0021
// off in the mean instead of 0.0017 (most of it their own rounding).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "mla_decode.h"
#include "mla_prefill.h"
#include "mla_score.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace chunk {

// O is rescaled (a round trip through TMEM that stalls PV, ~1.3 us) only when
// a row's maximum grows by more than 2^threshold over its reference.  P and
// the fp32 sums then reach 2^threshold; a float's relative precision does not
// depend on it.  bf16 P has fp32's range, so the threshold only has to keep
// sums and outputs finite (2^40 N |v| stays far below 2^127).  f16 P (e4m3
// cache) ends at 2^16.  A low first reference is common: a page of four sink
// tokens comes first, and with a threshold of 8 a window of 2048 tokens
// rescaled on 15 of its 34 pages.
template <bool kF8>
struct Rescale {
  static constexpr float kThreshold = kF8 ? 14.0f : 40.0f;
};
constexpr int kMaxClusters = 96;       // the combine's lanes take 3 clusters each

struct __align__(16) Ctrl {
  int4 unit[2][2];               // S: the unit whose queries land on q_bar (p0, p1, nrows, pos0), (h0, sp, skip, -)
  uint64_t kv_full[kMaxStages];
  uint64_t kv_empty[kMaxStages];
  uint64_t peer_kv[kMaxStages];  // S leader: the other S CTA's entry has landed
  uint64_t q_bar[2];             // query rows of the unit landed (alternating units)
  uint64_t s_full[kMaxSB];
  uint64_t s_empty[kMaxSB];         // S leader: both CTAs read the S buffer
  uint64_t q_full;               // S leader: queries in TMEM (both CTAs)
  uint64_t qs_full[2];           // e4m3: the unit's query scales (alternating units, as the ring may hold two)
  uint64_t q_part[3];            // bf16 pair: a part of the queries has been read
  uint64_t p_full[kMaxP];
  uint64_t p_empty[kMaxP];
  uint64_t peer_pv[kMaxP];       // O leader: the other O CTA is ready for PV of the page
  uint64_t v_full[4];            // e4m3: expanded pages
  uint64_t v_empty[4];
  uint64_t o_full;
  uint64_t o_empty;
  uint64_t resc_req;
  uint64_t resc_done;
  uint64_t ml_full;
  uint64_t ml_empty;
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t resc_page;
  uint32_t held[8];              // bf16 pair: what the S ring's slots hold (the producer's)
  int abort;
};
static_assert(sizeof(Ctrl) <= kCtrlBytes, "control block");

// One block of rows, as the schedule writes it.
struct Block {
  int32_t b;       // request
  int32_t row0;    // first row of the flattened [T * H]
  int32_t nrows;
  int32_t sp;      // virtual pages before the skip
  int32_t skip;    // real page = v + (v >= sp ? skip : 0)
  int32_t pos0;    // position of the first row's token (< 0: sees nothing)
  int32_t h0;      // head of the first row
  int32_t len;     // the request's length, clamped to the table
};
static_assert(sizeof(Block) == 32, "two 16-byte loads");

struct Params {
  const uint8_t* q_nope;
  const uint8_t* q_pe;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;      // [B + 1] first query token of each request; null: request b has tokens b*q_len ..
  uint8_t* out;
  float* lse;
  float* o_part;            // [2C][128 kCg][512]
  float* lse_part;          // [2C][128 kCg]
  int32_t* status;          // [4]
  int32_t* blkoff;          // [B + 1] first block of each request
  Block* blk;               // [NB]
  int32_t* prefix;          // [NB + 1] page prefix sums over blocks
  int32_t* cinfo;           // [C][4] slice start, end, first block, last block
  int32_t* cuts;            // [8] count, then [min(NB, C)][8] per block cut into pieces (any order): block, first
                            // cluster, last cluster, partial slot of the first piece, first row, rows
  int32_t B, H, q_len, T, NB, C, BR;  // BR = rows per block
  int32_t num_pages, max_pages, pt_stride;
  int32_t window, sinks;    // window 0: everything up to the row's own position
  int32_t unit_cost;        // schedule weight of starting a piece, in pages
  int32_t whole_pages;      // pages that a slice may have beyond the mean for blocks to stay whole
  float c2;                 // scale log2(e) (kv_scale), rounded once: scores in log2 units per product
  float kv_scale;
  uint64_t timeout_ns;
};

// ---------------------------------------------------------------- schedule
// One block of 1024 threads: the row blocks of every request, their page
// counts, and each cluster's slice of all pages.  Slices are cut in a
// weighted order (a piece of a block costs unit_cost pages to start), so that
// clusters with many short blocks get fewer pages.  A few blocks of about the
// same length get a cluster each instead: what a cut costs (fp32 partials, the
// combine) is more than what the even slices gain.
// Up to 256 requests and blocks (kSmall) every thread has one of each and all
// of it stays in shared memory; that form is half the code, and what a small
// call waits for here is mostly the first fetch of instructions.
constexpr int kSchedThreads = 1024;
constexpr int kSchedSmall = 256;    // threads, requests and blocks of the small form
constexpr int kSchedSmemNB = 8192;  // the other form: blocks and requests whose sums are kept in shared memory for
constexpr int kSchedSmemB = 2048;   // the searches

// The page of the last key that the block's last row sees.
__device__ __forceinline__ int last_page(const Block& k, int H) {
  const int pos1 = k.pos0 + (k.h0 + k.nrows - 1) / H;
  return (pos1 < 0 ? 0 : pos1) / kPage;
}

__device__ __forceinline__ int block_scan(int v, int* warp_tot, int carry) {  // inclusive, all threads
  const int tid = threadIdx.x;
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if ((tid & 31) >= o) v += t;
  }
  if ((tid & 31) == 31) warp_tot[tid >> 5] = v;
  __syncthreads();
  if (tid < 32) {
    int w = tid < static_cast<int>(blockDim.x >> 5) ? warp_tot[tid] : 0;
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, w, o);
      if (tid >= o) w += t;
    }
    warp_tot[tid] = w;
  }
  __syncthreads();
  return v + ((tid >> 5) ? warp_tot[(tid >> 5) - 1] : 0) + carry;
}

// The same for the small form, with one barrier; `tot` is written once per kernel.
__device__ __forceinline__ int block_scan_small(int v, int (&tot)[kSchedSmall / 32]) {
  const int tid = threadIdx.x;
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if ((tid & 31) >= o) v += t;
  }
  if ((tid & 31) == 31) tot[tid >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSchedSmall / 32; ++w) v += w < (tid >> 5) ? tot[w] : 0;
  return v;
}

template <bool kSmall>
__global__ void __launch_bounds__(kSmall ? kSchedSmall : kSchedThreads)
    mla_chunk_schedule_kernel(const __grid_constant__ Params p) {
  __shared__ int warp_tot[32];
  __shared__ __align__(16) int tot_b[kSchedSmall / 32], tot_n[kSchedSmall / 32];
  __shared__ int carry_s, ncuts, longest;
  // page prefix sums, first block of each request: copies for the searches (a
  // search through global memory waits ~0.7 us a step)
  __shared__ int32_t sp[(kSmall ? kSchedSmall : kSchedSmemNB) + 1];
  __shared__ int32_t sb[(kSmall ? kSchedSmall : kSchedSmemB) + 1];
  __shared__ int cb[kMaxClusters + 1];        // where the slices begin: page,
  __shared__ int cf[kMaxClusters + 1];        // and the block that holds it
  constexpr int kKept = kSmall ? kSchedSmall : 1;
  __shared__ int s_q0[kKept], s_nq[kKept], s_len[kKept];
  __shared__ int2 s_rows[kKept];              // a block's first row, rows
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  constexpr int nt = kSmall ? kSchedSmall : kSchedThreads;
  if (tid < 4) p.status[tid] = 0;
  if (tid == 0) carry_s = ncuts = longest = 0;
  __syncthreads();
  const bool sb_ok = kSmall || p.B <= kSchedSmemB, sp_ok = kSmall || p.NB <= kSchedSmemNB;
  // request b's query tokens [q0, q1); an invalid range is left out
  auto range = [&](int b, int& q0, int& q1) -> bool {
    if (!p.cu_q) {
      q0 = b * p.q_len;
      q1 = q0 + p.q_len;
      return true;
    }
    q0 = p.cu_q[b];
    q1 = p.cu_q[b + 1];
    if (q0 >= 0 && q1 >= q0 && q1 <= p.T && (b > 0 || q0 == 0)) return true;
    q0 = q1 = 0;
    return false;
  };
  // row blocks per request
  for (int base = 0; base < (kSmall ? 1 : p.B); base += nt) {
    const int b = base + tid;
    int nblk = 0;
    if (b < p.B) {
      const int L = p.seq_lens[b];
      int q0, q1;
      if (!range(b, q0, q1)) atomicOr(p.status, MLA_DEV_BAD_QUERY_RANGE);
      if (q1 > q0 && (L < q1 - q0 || L > p.max_pages * kPage)) atomicOr(p.status, MLA_DEV_BAD_SEQ_LEN);
      // (rows fit in 31 bits, rounded up in 32)
      nblk = static_cast<int>((static_cast<uint32_t>(q1 - q0) * static_cast<uint32_t>(p.H) + (p.BR - 1)) >>
                              (p.BR == 256 ? 8 : 7));
      if constexpr (kSmall) {
        s_q0[b] = q0;
        s_nq[b] = q1 - q0;
        s_len[b] = L;
      }
    }
    const int incl = kSmall ? block_scan_small(nblk, tot_b) : block_scan(nblk, warp_tot, carry_s);
    if (b < p.B) {
      const int v = incl < p.NB ? incl : p.NB;  // never beyond the arrays
      if (sb_ok) sb[b + 1] = v;
      else p.blkoff[b + 1] = v;
    }
    __syncthreads();
    if (tid == nt - 1) carry_s = incl <= p.NB ? incl : p.NB + 1;  // ranges that overlap could pass 32 bits
    if (!kSmall) __syncthreads();
  }
  if (tid == 0) {
    if (!sb_ok) p.blkoff[0] = 0;
    sb[0] = 0;
    if (!kSmall && carry_s > p.NB) atomicOr(p.status, MLA_DEV_BAD_QUERY_RANGE);
    if (!kSmall) carry_s = 0;
  }
  if (kSmall && tid == nt - 1 && carry_s > p.NB) atomicOr(p.status, MLA_DEV_BAD_QUERY_RANGE);
  __syncthreads();
  const int32_t* off = sb_ok ? sb : p.blkoff;
  const int nblocks = off[p.B];
  auto block_at = [&](int n) -> Block {
    int lo = 0, hi = p.B - 1;  // last request with off <= n
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= n) lo = mid; else hi = mid - 1;
    }
    int q0, nq, Lraw;
    if constexpr (kSmall) {
      q0 = s_q0[lo];
      nq = s_nq[lo];
      Lraw = s_len[lo];
    } else {
      int q1;
      range(lo, q0, q1);
      nq = q1 - q0;
      Lraw = p.seq_lens[lo];
    }
    // a request's rows fit in 31 bits (total_q * H does)
    const uint32_t r0 = static_cast<uint32_t>(n - off[lo]) * static_cast<uint32_t>(p.BR);  // within the request
    const uint32_t left = static_cast<uint32_t>(nq) * static_cast<uint32_t>(p.H) - r0;
    const int L = Lraw < 0 ? 0 : (Lraw > p.max_pages * kPage ? p.max_pages * kPage : Lraw);
    Block k;
    k.b = lo;
    k.row0 = static_cast<int32_t>(static_cast<uint32_t>(q0) * static_cast<uint32_t>(p.H) + r0);
    k.nrows = static_cast<int32_t>(left < static_cast<uint32_t>(p.BR) ? left : static_cast<uint32_t>(p.BR));
    const uint32_t i0 = r0 / static_cast<uint32_t>(p.H);
    k.h0 = static_cast<int32_t>(r0 - i0 * static_cast<uint32_t>(p.H));
    k.pos0 = L - nq + static_cast<int>(i0);
    k.len = L;
    const int last = last_page(k, p.H);  // at least one page, all of it masked if nothing is seen
    k.sp = last + 1;
    k.skip = 0;
    if (p.window > 0) {
      const int wp = k.pos0 + 1 > p.window ? (k.pos0 + 1 - p.window) / kPage : 0;  // page of the first row's first key
      const int ns = p.sinks / kPage + (p.sinks % kPage != 0);
      if (wp > ns) {
        k.sp = ns;
        k.skip = wp - ns;
      }
    }
    return k;
  };
  // each block's rows and pages
  int most = 0;
  for (int base = 0; base < (kSmall ? 1 : p.NB); base += nt) {
    const int n = base + tid;
    int np = 0;
    if (n < nblocks) {
      const Block k = block_at(n);
      np = last_page(k, p.H) + 1 - k.skip;
      most = np > most ? np : most;
      p.blk[n] = k;
      if constexpr (kSmall) s_rows[n] = make_int2(k.row0, k.nrows);
    }
    const int incl = kSmall ? block_scan_small(np, tot_n) : block_scan(np, warp_tot, carry_s);
    if (n < p.NB) {
      p.prefix[n + 1] = incl;
      if (sp_ok) sp[n + 1] = incl;
    }
    if (!kSmall) {
      __syncthreads();
      if (tid == nt - 1) carry_s = incl;
      __syncthreads();
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMax(&longest, most);
  if (tid == 0) {
    p.prefix[0] = 0;
    sp[0] = 0;
  }
  __syncthreads();
  const int32_t* pre = sp_ok ? sp : p.prefix;
  if (nblocks == 0) {
    for (int c = tid; c < p.C; c += nt)
      for (int k = 0; k < 4; ++k) p.cinfo[4 * c + k] = 0;
    if (tid == 0) p.cuts[0] = 0;
    return;
  }
  // slices: weighted position of block n's first page is pre[n] + unit_cost * (n + 1)
  const int64_t W = static_cast<int64_t>(pre[nblocks]) + static_cast<int64_t>(p.unit_cost) * nblocks;
  auto slice_at = [&](int c, int64_t x) {
    int lo = 0, hi = nblocks - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] + static_cast<int64_t>(p.unit_cost) * mid <= x) lo = mid; else hi = mid - 1;
    }
    const int64_t np = pre[lo + 1] - pre[lo];
    const int64_t off_p = x - pre[lo] - static_cast<int64_t>(p.unit_cost) * (lo + 1);
    cb[c] = off_p < 0 ? pre[lo] : (off_p >= np ? pre[lo + 1] : static_cast<int>(pre[lo] + off_p));
    cf[c] = off_p >= np ? lo + 1 : lo;  // (every block has a page)
  };
  const bool whole = nblocks <= p.C && longest <= pre[nblocks] / p.C + p.whole_pages;
  // W c / C without a 64-bit division: W = C quo + rem
  const int64_t quo = W < (static_cast<int64_t>(1) << 32) ? static_cast<uint32_t>(W) / static_cast<uint32_t>(p.C)
                                                          : W / p.C;
  const uint32_t rem = static_cast<uint32_t>(W - quo * p.C);
  for (int c = tid; c <= p.C; c += nt) {
    const int64_t x = quo * c + rem * static_cast<uint32_t>(c) / static_cast<uint32_t>(p.C);
    if (c == 0 || c == p.C || whole) {
      const int n = c == 0 ? 0 : (c == p.C || c > nblocks ? nblocks : c);
      cb[c] = pre[n];
      cf[c] = n;
    } else {
      slice_at(c, x);
    }
  }
  __syncthreads();
  for (int c = tid; c < p.C; c += nt) {
    const int s = cb[c], e = cb[c + 1];
    const int first = s < e ? cf[c] : 0, last = s < e ? cf[c + 1] - (pre[cf[c + 1]] == e ? 1 : 0) : 0;
    *reinterpret_cast<int4*>(p.cinfo + 4 * c) = make_int4(s, e, first, last);
    // the block that starts in this slice (or exactly with it) and goes on
    // behind it, if there is one: an entry of the combine's list
    if (s < e && pre[last + 1] > e && pre[last] >= s) {
      int lo = c, hi = p.C - 1;  // last cluster whose slice begins before the block's end
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cb[mid] < pre[last + 1]) lo = mid; else hi = mid - 1;
      }
      int2 rows;
      if constexpr (kSmall) rows = s_rows[last];
      else rows = make_int2(p.blk[last].row0, p.blk[last].nrows);
      int4* dst = reinterpret_cast<int4*>(p.cuts + 8 * (1 + atomicAdd(&ncuts, 1)));
      dst[0] = make_int4(last, c, lo, 2 * c + (first != last ? 1 : 0));
      dst[1] = make_int4(rows.x, rows.y, 0, 0);
    }
  }
  __syncthreads();
  if (tid == 0) p.cuts[0] = ncuts;
}

// One block's piece inside a cluster's slice.
struct Unit {
  int p0, p1, slot;  // virtual pages [p0, p1); slot < 0: the whole block
  Block k;
};

struct UnitIter {
  const Params* p;
  int s, e, n, nfirst, nlast, cid;
  __device__ void init(const Params& pp, int c) {
    p = &pp;
    cid = c;
    s = pp.cinfo[4 * c + 0];
    e = pp.cinfo[4 * c + 1];
    nfirst = pp.cinfo[4 * c + 2];
    nlast = pp.cinfo[4 * c + 3];
    n = nfirst;
  }
  __device__ bool next(Unit& u) {
    if (s >= e || n > nlast) return false;
    const int pb0 = p->prefix[n], pb1 = p->prefix[n + 1];
    u.p0 = (s > pb0 ? s : pb0) - pb0;
    u.p1 = (e < pb1 ? e : pb1) - pb0;
    const int4* src = reinterpret_cast<const int4*>(p->blk + n);
    const int4 a = src[0], b = src[1];
    u.k.b = a.x; u.k.row0 = a.y; u.k.nrows = a.z; u.k.sp = a.w;
    u.k.skip = b.x; u.k.pos0 = b.y; u.k.h0 = b.z; u.k.len = b.w;
    u.slot = (u.p0 > 0 || u.p1 < pb1 - pb0) ? 2 * cid + (n != nfirst ? 1 : 0) : -1;
    ++n;
    if (n <= nlast) {  // the next unit's lines into L1, for the CTA's other warps too
      prefetch_l1(p->blk + n);
      prefetch_l1(p->prefix + n + 1);
    }
    return true;
  }
};
__device__ __forceinline__ int real_page(const Block& k, int v) { return v + (v >= k.sp ? k.skip : 0); }

enum WaitTag : int {
  kWaitProdS = 101, kWaitProdO, kWaitQFull, kWaitKvS, kWaitPeerKv, kWaitSFull, kWaitPEmpty, kWaitMlEmpty, kWaitPage,
  kWaitRescDone, kWaitPeerPv, kWaitPvPrev, kWaitOFull, kWaitMlFull, kWaitSPrev, kWaitQEntry, kWaitPub, kWaitRaw,
  kWaitVEmpty, kWaitQScale
};

template <int kCg>
__device__ __forceinline__ void raise_timeout(const Params& p, Ctrl* ctrl, int tag, uint32_t j) {
  if (atomicCAS(p.status + 1, 0, tag) == 0) {
    p.status[2] = static_cast<int32_t>(j);
    p.status[3] = static_cast<int32_t>((cluster_id_x() << 16) | (cluster_ctarank() << 8) | (threadIdx.x >> 5));
  }
  atomicOr(p.status, MLA_DEV_TIMEOUT);
  for (uint32_t r = 0; r < 2 * kCg; ++r) st_cluster_u32(mapa(smem_u32(&ctrl->abort), r), 1u);
}

__device__ __forceinline__ int32_t read_page_id(const Params& p, int b, int pg) {
  const int32_t pid = __ldg(p.page_table + static_cast<int64_t>(b) * p.pt_stride + pg);
  if (pid < 0 || pid >= p.num_pages) {
    atomicOr(p.status, MLA_DEV_BAD_PAGE_ID);
    return 0;
  }
  return pid;
}

// Waits until the copies behind i phases of a ring's barriers have landed (bounded).
template <int kNSt>
__device__ __forceinline__ void drain_ring(Ctrl* ctrl, uint32_t i, uint64_t timeout_ns) {
  for (uint32_t q = 0; q < static_cast<uint32_t>(kNSt) && q < i; ++q) {
    const uint32_t last = i - 1 - ((i - 1 - q) % kNSt);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(&ctrl->kv_full[q]), (last / kNSt) & 1) && globaltimer_ns() - t0 < timeout_ns) {
    }
  }
}

// TMA producer of an S CTA: per unit its query rows (kQEntries ring entries,
// completing on q_bar), then its page of every tile (a unit's odd last tile
// has none for the second CTA: its barrier only gets an arrival).
//
// Where a page is one ring entry, every entry has its barriers (a query
// entry's complete by plain arrivals, so that the phases keep in step).  A
// bf16 pair's page is three entries, but has one barrier and frees its slots
// with its score tile: a commit and a wait per part kept the issuing warp
// busy for ~940 cycles per 768 cycles of MMAs (2815 a tile instead of 2304).
// So the slot of an entry is free once the tile of the page that it held is
// scored (s_full), or once the query part that it held is in TMEM (q_part).
template <bool kF8, int kCg>
__device__ void produce_s(const Params& p, Ctrl* ctrl, uint8_t* ring, const CUtensorMap* tm_s, const CUtensorMap* tm_pe,
                          const CUtensorMap* tm_qn, const CUtensorMap* tm_qp, int cid, int pr) {
  using C = Cfg<kF8, kCg>;
  volatile int* abort = &ctrl->abort;
  UnitIter it;
  it.init(p, cid);
  Unit u;
  uint32_t i = 0, un = 0;
  bool ok = true;
  uint32_t bar = 0, jt = 0;  // jt: tiles
  uint32_t scored = 0;       // tiles known to be scored
  uint8_t* slot = nullptr;
  // a free slot for entry i; `held`: what the entry will be, 4 unit + part of
  // the queries or 4 tile + 3 (waiting for a tile only until it is known to be
  // scored also keeps the parity right: two tiles later it would be wrong)
  auto acquire = [&](uint32_t held) -> bool {
    const int st = static_cast<int>(i % C::kNStS);
    slot = ring + st * C::kSlotS;
    if constexpr (C::kParts == 3) {
      if (i >= static_cast<uint32_t>(C::kNStS)) {
        const uint32_t was = ctrl->held[st], k = was >> 2;
        if ((was & 3u) == 3u) {
          if (k >= scored && !mbar_wait(smem_u32(&ctrl->s_full[k % C::kNSB]), (k / C::kNSB) & 1, abort, p.timeout_ns))
            return false;
          scored = k >= scored ? k + 1 : scored;
        } else if (!mbar_wait(smem_u32(&ctrl->q_part[was & 3u]), k & 1, abort, p.timeout_ns)) {
          return false;
        }
      }
      ctrl->held[st] = held;
      return true;
    } else {
      bar = smem_u32(&ctrl->kv_full[st]);
      return mbar_wait(smem_u32(&ctrl->kv_empty[st]), ((i / C::kNStS) & 1) ^ 1, abort, p.timeout_ns);
    }
  };
  uint32_t qloaded = 0;
  // the next unit's query rows are pulled into L2 a few pages ahead
  UnitIter ahead;
  ahead.init(p, cid);
  Unit nx;
  bool have_next = ahead.next(nx);
  while (ok && it.next(u)) {
    const uint32_t qbar = smem_u32(&ctrl->q_bar[un & 1]);
    const int row0 = u.k.row0 + pr * kRows;
    const int qe = C::q_entries(u.k.nrows);
    have_next = have_next && ahead.next(nx);
    const int pf = u.p1 - 4 * kCg > u.p0 ? u.p0 + (u.p1 - 4 * kCg - u.p0) / kCg * kCg : u.p0;
    for (int e = 0; e < qe; ++e) {
      if (!acquire(4 * un + static_cast<uint32_t>(e) / 2)) {
        ok = false;
        break;
      }
      if (e == 0) {
        ctrl->unit[un & 1][0] = make_int4(u.p0, u.p1, u.k.nrows, u.k.pos0);
        ctrl->unit[un & 1][1] = make_int4(u.k.h0, u.k.sp, u.k.skip, 0);
        mbar_expect_tx(qbar, static_cast<uint32_t>(C::kParts == 3 ? kRows * 1152 : qe * C::kQRows * 1152));
        qloaded = un + 1;
        if constexpr (C::kParts == 3)
          tma_load_2d(smem_u32(ring + C::kQPeOff + (un & 1) * C::kQPeTile), tm_qp, 0, row0, qbar);
      }
      if constexpr (C::kParts == 1) mbar_arrive(bar);
      if constexpr (C::kParts == 3) {
        // boxes 3 (e / 2) .. of 64 rows; the third part's last box would be
        // past the map's 8: it reads zeros, which count as copied bytes too,
        // so its two boxes come one by one
        const int row = row0 + 64 * (e % 2), part = e / 2;
        if (part < 2) {
          tma_load_3d(smem_u32(slot), tm_qn, 0, row, 3 * part, qbar);
        } else {
          tma_load_2d(smem_u32(slot), tm_pe, 64 * 6, row, qbar);
          tma_load_2d(smem_u32(slot + C::kBox), tm_pe, 64 * 7, row, qbar);
        }
      } else {
        const int row = row0 + C::kQRows * e;
        tma_load_3d(smem_u32(slot), tm_qn, 0, row, 0, qbar);
        tma_load_2d(smem_u32(slot + C::kQRows * 128 * 8), tm_qp, 0, row, qbar);
      }
      ++i;
    }
    ++un;
    for (int vt = u.p0; vt < u.p1 && ok; vt += kCg, ++jt) {
      if (have_next && vt == pf) {
        const int64_t r0 = static_cast<int64_t>(nx.k.row0) + pr * kRows;
        const int left = nx.k.nrows - pr * kRows, n = left < kRows ? left : kRows;
        if (n > 0) {
          prefetch_l2_bulk(p.q_nope + r0 * kDL * 2, static_cast<uint32_t>(n) * kDL * 2);
          prefetch_l2_bulk(p.q_pe + r0 * kDR * 2, static_cast<uint32_t>(n) * kDR * 2);
        }
      }
      const int v = vt + pr;
      const bool have = kCg == 1 || v < u.p1;
      const int y = have ? read_page_id(p, u.k.b, real_page(u.k, v)) * kPage : 0;
      for (int part = 0; part < C::kParts; ++part) {
        if (!acquire(4 * jt + 3)) {
          ok = false;
          break;
        }
        if constexpr (C::kParts == 3) bar = smem_u32(&ctrl->kv_full[jt % C::kNTile]);
        if (have) {
          if (part == 0) mbar_expect_tx(bar, static_cast<uint32_t>(C::kParts * C::kSlotS));
          tma_load_3d(smem_u32(slot), tm_s, 0, y, part * C::kPartBoxes, bar);
          if constexpr (kF8) tma_load_2d(smem_u32(slot + C::kSBoxes * C::kBox), tm_pe, kDL, y, bar);
        } else if (part == 0) {
          mbar_arrive(bar);
        }
        ++i;
      }
    }
  }
  if (!ok) raise_timeout<kCg>(p, ctrl, kWaitProdS, i);
  drain_ring<C::kNTile>(ctrl, C::kParts == 3 ? jt : i, p.timeout_ns);
  // the last unit's query rows: a unit cut short by a timeout may not have
  // armed all its bytes, so this wait is bounded too
  if (qloaded) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(smem_u32(&ctrl->q_bar[(qloaded - 1) & 1]), ((qloaded - 1) >> 1) & 1) &&
           globaltimer_ns() - t0 < p.timeout_ns) {
    }
  }
}

// TMA producer of an O CTA: its latent dimensions of every page.
template <bool kF8, int kCg>
__device__ void produce_o(const Params& p, Ctrl* ctrl, uint8_t* ring, const CUtensorMap* tm_o, int cid, int pr) {
  using C = Cfg<kF8, kCg>;
  volatile int* abort = &ctrl->abort;
  UnitIter it;
  it.init(p, cid);
  Unit u;
  uint32_t i = 0;
  bool ok = true;
  while (ok && it.next(u)) {
    for (int v = u.p0; v < u.p1; ++v) {
      const int y = read_page_id(p, u.k.b, real_page(u.k, v)) * kPage;
      const int st = static_cast<int>(i % C::kNStO);
      // with as many P slots as V slots, P's barrier tells both
      const uint32_t empty = smem_u32(C::kVByP ? &ctrl->p_empty[st] : &ctrl->kv_empty[st]);
      if (!mbar_wait(empty, ((i / C::kNStO) & 1) ^ 1, abort, p.timeout_ns)) {
        raise_timeout<kCg>(p, ctrl, kWaitProdO, i);
        ok = false;
        break;
      }
      const uint32_t bar = smem_u32(&ctrl->kv_full[st]);
      mbar_expect_tx(bar, static_cast<uint32_t>(C::kSlotO));
      tma_load_3d(smem_u32(ring + st * C::kSlotO), tm_o, 0, y, pr * (kF8 ? C::kRawBoxes : C::kVBoxes), bar);
      ++i;
    }
  }
  drain_ring<C::kNStO>(ctrl, i, p.timeout_ns);
}

// Column c of O is latent dimension c, or with kCg = 2 (each PV MMA's N = 256
// is half from each CTA of the pair) 256 ((c / 128) % 2) + 128 (c / 256) + c % 128.
template <int kCg>
__device__ __forceinline__ int dim_of(int c) {
  return kCg == 1 ? c : (((c >> 7) & 1) * 256 + (c >> 8) * 128 + (c & 127));
}

// Writes a row's log-sum-exp (of the whole block's keys, or of a piece's) and
// returns the factor of its outputs.
template <bool kF8>
__device__ __forceinline__ float store_lse(const Params& p, const Unit& u, int br, bool mine, float m_log2, float l) {
  const float inv_l = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // a NaN sum stays NaN
  if (mine && br < u.k.nrows && u.slot < 2 * p.C) {
    const float lse_v = l > 0.f ? (m_log2 + __log2f(l)) * kLn2 : (l == 0.f ? -INFINITY : l);
    if (u.slot < 0) p.lse[static_cast<int64_t>(u.k.row0) + br] = lse_v;
    else p.lse_part[static_cast<int64_t>(u.slot) * p.BR + br] = lse_v;
  }
  return kF8 ? p.kv_scale * 256.f * inv_l : inv_l;  // e4m3 values are in f16 as value / 256
}

// A warp's 32 rows br0 .. (TMEM lanes), columns [c0, c0 + 256), by way of
// shared memory: boxes of 32 rows x 64 bytes (64-byte swizzle), kBufs in turn,
// that TMA writes.  (A lane's own stores to its row take a line each: a block's
// bf16 outputs took 4.9 us that way, 2.5 this way, and O is not free for the
// next block before that.)
template <bool kF8, int kCg>
__device__ __forceinline__ void store_staged(const Params& p, const Unit& u, int br0, int c0, uint32_t taddr, float f,
                                             uint8_t* stage, const CUtensorMap* map) {
  constexpr int kBufs = Cfg<kF8, kCg>::kStage > 2048 ? 2 : 1;
  const int lane = threadIdx.x & 31;
  const bool whole = u.slot < 0;
  const int y = whole ? u.k.row0 + br0 : u.slot * p.BR + br0;
  uint32_t v[2][16];
  tmem_ld16(taddr + c0, v[0]);
  tmem_ld16(taddr + c0 + 16, v[1]);
#pragma unroll 1
  for (int s = 0; s < 8; ++s) {
    tmem_wait_ld_tie(v[0]);
    tmem_wait_ld_tie(v[1]);
    float x[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(v[k >> 4][k & 15]) * f;
    if (s < 7) {
      tmem_ld16(taddr + c0 + 32 * s + 32, v[0]);
      tmem_ld16(taddr + c0 + 32 * s + 48, v[1]);
    }
    const int dim = dim_of<kCg>(c0 + 32 * s);
    auto put = [&](const uint32_t (&w)[16], int buf, int xdim, bool wait) {
      if (wait) {
        if (lane == 0) bulk_wait_read<kBufs - 1>();
        __syncwarp();
      }
      uint8_t* row = stage + buf * 2048 + lane * 64;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(row + ((c ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      fence_proxy_async_cta();
      __syncwarp();
      if (lane == 0) tma_store_2d(map, smem_u32(stage + buf * 2048), xdim, y);
    };
    uint32_t w[16];
    if (whole) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      put(w, s % kBufs, dim, s >= kBufs);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(x[16 * h + k]);
        put(w, h % kBufs, dim + 16 * h, 2 * s + h >= kBufs);
      }
    }
  }
}

// The same for one row from the thread's own stores, columns [c0, c1): bf16
// out for a whole block, fp32 partials (normalised O) for a piece.
template <bool kF8, int kCg>
__device__ __forceinline__ void store_row(const Params& p, const Unit& u, int br, int c0, int c1, uint32_t taddr,
                                          float f) {
  if (u.slot >= 2 * p.C) {  // cannot happen; a bad schedule never writes out of range
    atomicOr(p.status, MLA_DEV_INTERNAL);
    return;
  }
  const bool real = br < u.k.nrows;
  const int64_t orow = static_cast<int64_t>(u.k.row0) + br;
  const int64_t prow = static_cast<int64_t>(u.slot) * p.BR + br;
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    const int dim = dim_of<kCg>(c);
    uint32_t v[2][16];
    tmem_ld16(taddr + c, v[0]);
    tmem_ld16(taddr + c + 16, v[1]);
    tmem_wait_ld_tie(v[0]);
    tmem_wait_ld_tie(v[1]);
    if (!real) continue;
    if (u.slot < 0) {
      uint8_t* dst = p.out + (orow * kDL + dim) * 2;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const __nv_bfloat162 b2 =
              __floats2bfloat162_rn(__uint_as_float(v[q][2 * k]) * f, __uint_as_float(v[q][2 * k + 1]) * f);
          w[k] = *reinterpret_cast<const uint32_t*>(&b2);
        }
        stg_v8(dst + 32 * q, w);
      }
    } else {
      float* dst = p.o_part + prow * kDL + dim;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(v[q][8 * k + e]) * f);
          stg_v8(dst + 16 * q + 8 * k, w);
        }
    }
  }
}

// --------------------------------------------------------------- attention
template <bool kF8, int kCg>
__global__ void __launch_bounds__(kThreads, 1)
    mla_chunk_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_s,
                     const __grid_constant__ CUtensorMap tm_o, const __grid_constant__ CUtensorMap tm_pe,
                     const __grid_constant__ CUtensorMap tm_qn, const __grid_constant__ CUtensorMap tm_qp,
                     const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ CUtensorMap tm_part) {
  using C = Cfg<kF8, kCg>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* data = smem_raw;
  if ((smem_u32(data) & 1023u) != 0u) {  // the same in every CTA; swizzled tiles need it
    griddep_wait();
    if (threadIdx.x == 0) atomicOr(p.status, MLA_DEV_INTERNAL);
    return;
  }
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(data + ((C::kData + 15) & ~15));
  // ranks 0 .. kCg - 1: S CTAs; kCg .. 2 kCg - 1: O CTAs; pr: place in the pair
  const uint32_t rank = cluster_ctarank();
  const bool role_s = rank < kCg;
  const int pr = static_cast<int>(rank % kCg);
  const bool leader = pr == 0;
  const int cid = static_cast<int>(cluster_id_x());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr uint16_t kMaskS = (1u << kCg) - 1u, kMaskO = kMaskS << kCg, kMaskAll = kMaskS | kMaskO;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(smem_u32(&ctrl->kv_full[i]), 1);
      mbar_init(smem_u32(&ctrl->kv_empty[i]), (!role_s && kF8) ? 8 : 1);  // e4m3 O CTA: the eight expanding warps
      mbar_init(smem_u32(&ctrl->peer_kv[i]), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctrl->q_bar[i]), 1);
    for (int i = 0; i < C::kNSB; ++i) {
      mbar_init(smem_u32(&ctrl->s_full[i]), 1);
      // the warps that read the tile: one group's four, or both groups' of both CTAs
      mbar_init(smem_u32(&ctrl->s_empty[i]), kCg == 1 ? 4 : 16);
    }
    mbar_init(smem_u32(&ctrl->q_full), 8 * kCg);
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&ctrl->q_part[i]), 8);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&ctrl->qs_full[i]), 2);
    for (int i = 0; i < kMaxP; ++i) {
      mbar_init(smem_u32(&ctrl->p_full[i]), 1);
      mbar_init(smem_u32(&ctrl->p_empty[i]), 1);
      mbar_init(smem_u32(&ctrl->peer_pv[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&ctrl->v_full[i]), 8);
      mbar_init(smem_u32(&ctrl->v_empty[i]), 1);
    }
    mbar_init(smem_u32(&ctrl->o_full), 1);
    mbar_init(smem_u32(&ctrl->o_empty), C::kCorrWarps);
    mbar_init(smem_u32(&ctrl->resc_req), 1);
    mbar_init(smem_u32(&ctrl->resc_done), C::kCorrWarps);
    mbar_init(smem_u32(&ctrl->ml_full), kCg == 1 ? 8 : 1);  // a pair: by bytes
    mbar_init(smem_u32(&ctrl->ml_empty), C::kCorrWarps);
    mbar_init(smem_u32(&ctrl->drain), 1);
    ctrl->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(role_s ? &tm_s : &tm_o);
    if (role_s) tma_prefetch_desc(&tm_qn);
    if (role_s) tma_prefetch_desc(&tm_qp);
    if (role_s && kF8) tma_prefetch_desc(&tm_pe);
  }
  if (role_s && threadIdx.x >= 128)  // page references: no page yet
    for (int i = threadIdx.x - 128; i < 4 * kRows; i += kThreads - 128)
      reinterpret_cast<uint64_t*>(data + C::kPubOff)[i] = 0ull;
  __syncthreads();
  cluster_sync();  // barriers initialised before any remote arrival; both CTAs of a pair here before the pair's alloc
  if (warp == 2) {
    tmem_alloc_cg<kCg>(smem_u32(&ctrl->tmem_base), 512);
    tmem_relinquish_cg<kCg>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's TMEM exists before the leader's first MMA writes it
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = ctrl->tmem_base;
  volatile int* abort = &ctrl->abort;

  if (role_s) {
    // =========================== S CTA ===========================
    uint8_t* ring = data;
    if (warp == 0) {
      if (lane == 0) produce_s<kF8, kCg>(p, ctrl, ring, &tm_s, &tm_pe, &tm_qn, &tm_qp, cid, pr);
    } else if (warp == 1) {
      // The leader's warp issues QK for the pair (the whole warp runs the
      // loop, one elected lane issues); the other CTA's warp passes on that
      // its pages have landed.  Every barrier's every phase is waited for, the
      // query entries' too, so that none is ever missed.
      UnitIter it;
      it.init(p, cid);
      Unit u;
      uint32_t i = 0, j = 0, un = 0;  // ring entries, tiles, units
      bool ok = true;
      int why = 0;
      // barrier n (an entry's, a tile's) of this CTA and, for the leader, of
      // the other one; `extra` is polled along with them (0: nothing)
      auto landed = [&](uint32_t n, uint32_t extra, uint32_t extra_parity) -> bool {
        const int st = static_cast<int>(n % C::kNTile);
        const uint32_t ph = (n / C::kNTile) & 1;
        if (!mbar_wait_all_warp(smem_u32(&ctrl->kv_full[st]), ph,
                                kCg == 2 && leader ? smem_u32(&ctrl->peer_kv[st]) : 0u, ph, extra, extra_parity, 0u, 0u,
                                abort, p.timeout_ns)) {
          why = kWaitKvS;
          return false;
        }
        if (kCg == 2 && !leader && lane == 0) mbar_arrive_remote(mapa(smem_u32(&ctrl->peer_kv[st]), 0));
        return true;
      };
      while (ok && it.next(u)) {
        const int qe = C::q_entries(u.k.nrows);
        if constexpr (C::kParts == 3) {
          i += qe;
        } else {
          for (int e = 0; e < qe && ok; ++e, ++i) ok = landed(i, 0u, 0u);
          if (!ok) break;
        }
        if (leader) {
          if (!mbar_wait_warp(smem_u32(&ctrl->q_full), un & 1, abort, p.timeout_ns)) {
            ok = false;
            why = kWaitQFull;
            break;
          }
          if constexpr (kF8 && kCg == 2) mbar_acquire_shared(smem_u32(&ctrl->q_full), un & 1);  // both rope tiles
          if (lane == 0 && C::kParts == 1)  // the query entries' slots go back to the producers
            for (int e = qe; e > 0; --e) {
              const uint32_t bar = smem_u32(&ctrl->kv_empty[(i - e) % C::kNStS]);
              mbar_arrive(bar);
              if (kCg == 2) mbar_arrive_remote(mapa(bar, 1));
            }
          __syncwarp();
        }
        const uint32_t qpe = smem_u32(ring + C::kQPeOff + (kF8 ? 0 : (un & 1) * C::kQPeTile));
        ++un;
        for (int vt = u.p0; vt < u.p1; vt += kCg, ++j, i += C::kParts) {
          const int sb = static_cast<int>(j % C::kNSB);
          const uint32_t dcol = tmem + C::kSCol0 + sb * C::kTileCols;
          if (!landed(C::kParts == 3 ? j : i, leader ? smem_u32(&ctrl->s_empty[sb]) : 0u, ((j / C::kNSB) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (!leader) continue;
          tc_fence_after();
          if constexpr (!kF8) {
#pragma unroll
            for (int part = 0; part < C::kParts; ++part) {
              const uint32_t slot_addr = smem_u32(ring + ((i + part) % C::kNStS) * C::kSlotS);
              const uint64_t dlat = smem_desc(slot_addr, 16, 1024, kSwizzle128B);
#pragma unroll
              for (int d = 0; d < C::kPartBoxes; ++d)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int box = part * C::kPartBoxes + d;
                  const uint64_t db = dlat + static_cast<uint64_t>(d * (C::kBox >> 4) + k * 2);
                  if (C::kPeSmem && box == 8)
                    mma_ss_cg<kCg>(dcol, smem_desc(qpe, 16, 1024, kSwizzle128B) + static_cast<uint64_t>(k * 2), db,
                                   C::kIdescQK, 1u);
                  else
                    mma_ts_cg<false, kCg>(dcol, tmem + box * 32 + k * 8, db, C::kIdescQK, (box | k) ? 1u : 0u);
                }
            }
          } else {
            const uint32_t slot_addr = smem_u32(ring + (i % C::kNStS) * C::kSlotS);
            const uint64_t dlat = smem_desc(slot_addr, 16, 1024, kSwizzle128B);
            const uint64_t dpe = smem_desc(slot_addr + C::kSBoxes * C::kBox, 16, 512, kSwizzle64B);
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              const uint32_t qcol = tmem + (term ? C::kQLoCol : 0u);
#pragma unroll
              for (int d = 0; d < 4; ++d)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma_ts_cg<true, kCg>(dcol, qcol + d * 32 + k * 8,
                                       dlat + static_cast<uint64_t>(d * (C::kBox >> 4) + k * 2), C::kIdescQK,
                                       (term | d | k) ? 1u : 0u);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if constexpr (C::kPeSmem)
                  mma_ss_f8_cg<kCg>(dcol, smem_desc(qpe + term * C::kQPeTile, 128, 512, kSwizzleNone) +
                                              static_cast<uint64_t>(k * (256 >> 4)),
                                    dpe + static_cast<uint64_t>(k * 2), C::kIdescQK, 1u);
                else
                  mma_ts_cg<true, kCg>(dcol, qcol + 128 + k * 8, dpe + static_cast<uint64_t>(k * 2), C::kIdescQK, 1u);
              }
            }
          }
          if (C::kParts == 1) mma_commit_cg<kCg>(smem_u32(&ctrl->kv_empty[i % C::kNStS]), kMaskS);
          mma_commit_cg<kCg>(smem_u32(&ctrl->s_full[sb]), kMaskS);
        }
      }
      if (!ok && lane == 0) raise_timeout<kCg>(p, ctrl, why, j);
      __syncwarp();
      if (leader) {
        mma_commit_cg<kCg>(smem_u32(&ctrl->drain), static_cast<uint16_t>(1u << rank));
        if (lane == 0) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(&ctrl->drain), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
          }
        }
      }
      __syncwarp();
    } else if (kF8 && warp < 4) {
      // ---- warps 2 and 3: every row's query scale, while the row warps are
      // still at the unit before (two buffers: the next unit's queries come
      // into the ring after this unit's are in TMEM)
      UnitIter it;
      it.init(p, cid);
      Unit u;
      uint32_t i = 0, un = 0;
      bool ok = true;
      float* scales = reinterpret_cast<float*>(data + C::kQsOff);
      while (it.next(u)) {
        ok = mbar_wait_warp<false, true>(smem_u32(&ctrl->q_bar[un & 1]), (un >> 1) & 1, abort, p.timeout_ns);
        if (!ok) break;
        const int qe = C::q_entries(u.k.nrows);
        for (int r = (warp - 2) * 64 + lane; r < (warp - 1) * 64; r += 32)
          if (r < qe * C::kQRows) scales[(un & 1) * kRows + r] = q_row_scale<kCg>(ring, i, r);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctrl->qs_full[un & 1]));
        i += qe + C::kParts * static_cast<uint32_t>((u.p1 - u.p0 + kCg - 1) / kCg);
        ++un;
      }
      if (!ok && lane == 0) raise_timeout<kCg>(p, ctrl, kWaitQScale, un);
    } else if (warp >= 4) {
      // ---- softmax: thread r of group gg (warps 4-7: 0, warps 8-11: 1) takes
      // row r of this CTA, the groups alternate pages (tiles of one page, or
      // one page each of a pair's tile of two).  A page's reference
      // is the previous page's, raised to the page's maximum where that
      // exceeds it by more than the threshold, so references depend on the
      // data alone; each group keeps its partial sum in its latest frame.
      const int r = (warp & 3) * 32 + lane;
      const int gg = (warp - 4) >> 2;
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t orank = kCg + pr;
      const uint32_t p_remote = mapa(smem_u32(data), orank);
      const uint32_t ref_remote = mapa(smem_u32(data + C::kRefOff), orank);
      const uint32_t flag_remote = mapa(smem_u32(data + C::kFlagOff), orank);
      const uint32_t mlfull_remote = mapa(smem_u32(&ctrl->ml_full), orank);
      volatile uint64_t* pub = reinterpret_cast<volatile uint64_t*>(data + C::kPubOff);
      const int br = pr * kRows + r;  // row in the block
      UnitIter it;
      it.init(p, cid);
      Unit u;
      uint32_t i = 0, jt = 0, j0 = 0, un = 0;  // ring entries, tiles, pages of earlier units, units
      uint32_t j = 0;                          // page
      bool ok = true;
      int why = 0;
      // units come from the producer with their queries: loads of the schedule
      // would stand between a unit's last P and the next one's queries
      const uint32_t units = it.s < it.e ? static_cast<uint32_t>(it.nlast - it.nfirst + 1) : 0u;
      while (ok && un < units) {
        // the unit's queries replace the previous unit's in TMEM once every
        // QK of that unit is done: the S of its last tile has landed
        if (jt > 0 && !mbar_wait_warp<false, true>(smem_u32(&ctrl->s_full[(jt - 1) % C::kNSB]),
                                                   ((jt - 1) / C::kNSB) & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitSPrev;
          break;
        }
        if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->q_bar[un & 1]), (un >> 1) & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitQEntry;
          break;
        }
        {
          const int4 x = ctrl->unit[un & 1][0], y = ctrl->unit[un & 1][1];
          u.p0 = x.x; u.p1 = x.y; u.k.nrows = x.z; u.k.pos0 = x.w;
          u.k.h0 = y.x; u.k.sp = y.y; u.k.skip = y.z;
        }
        if (kF8 && !mbar_wait_warp<false, true>(smem_u32(&ctrl->qs_full[un & 1]), (un >> 1) & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitQScale;
          break;
        }
        float qs = 1.f;
        const int qe = C::q_entries(u.k.nrows);
        // (rows past the block's entries keep what TMEM holds: their results go nowhere)
        const bool loads = (warp & 3) * 32 < qe / C::kParts * C::kQRows;  // one answer per warp
        if (!loads) {
        } else if constexpr (kF8) {
          uint8_t* pe_tile = data + C::kQPeOff;
          qs = reinterpret_cast<const float*>(data + C::kQsOff)[(un & 1) * kRows + r];
          q_row_e4m3<kCg>(ring, i, r, tmem + lane_base, pe_tile, gg == 0 ? 0 : 5, gg == 0 ? 5 : 9, qs);
        } else if constexpr (C::kParts == 3) {
          auto part_read = [&](int part) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctrl->q_part[part]));
          };
          q_row_bf16<kCg, 12>(ring, i, r, tmem + lane_base, 12 * gg);
          part_read(0);
          q_row_bf16<kCg, 12>(ring, i, r, tmem + lane_base, 24 + 12 * gg);
          part_read(1);
          q_row_bf16<kCg, 8>(ring, i, r, tmem + lane_base, 48 + 8 * gg);
          part_read(2);
          tmem_wait_st();
        } else {
          q_row_bf16<kCg, 36>(ring, i, r, tmem + lane_base, 36 * gg);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {  // (an e4m3 pair's rope tile is ordinary stores that the leader's MMAs read)
          if (kCg == 2 && kF8) mbar_arrive_shared(mapa(smem_u32(&ctrl->q_full), 0));
          else if (kCg == 2) mbar_arrive_remote(mapa(smem_u32(&ctrl->q_full), 0));
          else mbar_arrive(smem_u32(&ctrl->q_full));
        }
        i += qe + C::kParts * static_cast<uint32_t>((u.p1 - u.p0 + kCg - 1) / kCg);
        // qs is a power of two, 2^-107 of a row of zeros: a product that small
        // counts as the least normal value (its scores are below 2^-90 in
        // either case), as 0 would turn masked scores into NaN
        float c2 = kF8 ? p.c2 * qs : p.c2;
        if (kF8 && c2 < 0x1p-126f) c2 = 0x1p-126f;
        const bool real = br < u.k.nrows;
        // padding rows follow the block's last row (their results go nowhere)
        const int pos = u.k.pos0 + (u.k.h0 + (real ? br : u.k.nrows - 1)) / p.H;
        const int nvis = pos + 1;                                                     // sees t < nvis ...
        const int lo = p.window > 0 && nvis > p.window ? nvis - p.window : 0;         // ... and t >= lo or t < sinks
        float m_run = kMinusBig, l = 0.f;
        for (int vt = u.p0; vt < u.p1; vt += kCg, ++jt) {
          if (kCg == 1 && (jt & 1u) != static_cast<uint32_t>(gg)) continue;
          const int vp = kCg == 1 ? vt : vt + gg;
          j = j0 + static_cast<uint32_t>(vp - u.p0);
          const int sb = static_cast<int>(jt % C::kNSB);
          if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->s_full[sb]), (jt / C::kNSB) & 1, abort, p.timeout_ns)) {
            ok = false;
            why = kWaitSFull;
            break;
          }
          if (kCg == 2 && vp >= u.p1) {  // an odd unit's last tile holds one page
            if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&ctrl->s_empty[sb]), 0));
            continue;
          }
          tc_fence_after();
          uint32_t v[4][16];
          float red[4];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            tmem_ld16_max(tmem + lane_base + C::kSCol0 + sb * C::kTileCols + (kCg == 2 ? gg * 64 : 0) + q4 * 16, v[q4],
                          red[q4]);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) tmem_wait_ld_tie(v[q4], red[q4]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (kCg == 2) mbar_arrive_remote(mapa(smem_u32(&ctrl->s_empty[sb]), 0));
            else mbar_arrive(smem_u32(&ctrl->s_empty[sb]));
          }
          const int t0 = real_page(u.k, vp) * kPage;
          const bool full = t0 + kPage <= nvis && (t0 >= lo || t0 + kPage <= p.sinks);
          // the page's keys [a, z) and [0, s) are seen
          const int z = nvis - t0, a = lo - t0, s = p.sinks - t0;
#define MLA_S(t) __uint_as_float(v[(t) >> 4][(t) & 15])
          float m4[4] = {red[0], red[1], red[2], red[3]};
          if (!full) {
            // unseen keys become -inf here (their P is then exactly 0), so
            // that whatever an unused slot holds, even NaN, never counts
            m4[0] = m4[1] = m4[2] = m4[3] = -INFINITY;
#pragma unroll
            for (int t = 0; t < 64; ++t) {
              const float x = (t < z && (t >= a || t < s)) ? MLA_S(t) : -INFINITY;
              v[t >> 4][t & 15] = __float_as_uint(x);
              m4[t & 3] = fmaxf(m4[t & 3], x);
            }
          }
          const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
          float m_ref = m_run;
          float m_prev = kMinusBig;
          if (vp != u.p0) {
            volatile uint64_t* pe = pub + ((j - 1u) & 3u) * kRows + r;
            uint64_t pv = *pe;
            if (static_cast<uint32_t>(pv >> 32) != j) {
              const uint64_t t_start = globaltimer_ns();
              while (static_cast<uint32_t>((pv = *pe) >> 32) != j) {
                if (*abort || globaltimer_ns() - t_start > p.timeout_ns) break;
              }
            }
            if (__any_sync(0xffffffffu, static_cast<uint32_t>(pv >> 32) != j)) {
              ok = false;
              why = kWaitPub;
              break;
            }
            m_prev = __uint_as_float(static_cast<uint32_t>(pv));
            m_ref = fmaxf(m_ref, m_prev);
          }
          if (mx > m_ref + Rescale<kF8>::kThreshold) m_ref = mx;
          pub[(j & 3u) * kRows + r] = (static_cast<uint64_t>(j + 1u) << 32) | __float_as_uint(m_ref);
          // a row that has seen nothing yet holds O = 0 in any frame
          const bool rose = vp != u.p0 && m_ref > m_prev && m_prev > kMinusBig;
          const float o_scale = rose ? ex2_approx(m_prev - m_ref) : 1.f;
          const uint32_t rose_mask = __ballot_sync(0xffffffffu, rose && real);
          l *= ex2_approx(m_run - m_ref);
          m_run = m_ref;
          const int ps = static_cast<int>(j % C::kNP);
          const uint32_t bar = mapa(smem_u32(&ctrl->p_full[ps]), orank);
          const uint32_t prow = p_remote + ps * C::kPBytes + (r >> 3) * C::kPSbo + (r & 7) * 16;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
          uint4 pw[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x = ex2_approx(fmaf(MLA_S(8 * c + 2 * k), c2, -m_ref));
              const float y = ex2_approx(fmaf(MLA_S(8 * c + 2 * k + 1), c2, -m_ref));
              s4[k] += x + y;  // the sum takes P before its rounding (bf16: half a step is 2^-8 relative, either sign)
              if constexpr (kF8) {  // f16, as the expanded values: 2^-11 relative, 2^-25 absolute at least
                const __half2 h2 = __floats2half2_rn(x, y);
                w[k] = *reinterpret_cast<const uint32_t*>(&h2);
              } else {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(x, y);
                w[k] = *reinterpret_cast<const uint32_t*>(&b2);
              }
            }
            pw[c] = make_uint4(w[0], w[1], w[2], w[3]);
          }
#undef MLA_S
          if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->p_empty[ps]), ((j / C::kNP) & 1) ^ 1, abort, p.timeout_ns)) {
            ok = false;
            why = kWaitPEmpty;
            break;
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) st_async_v4(prow + c * C::kPLbo, pw[c], bar);
          st_async_b32(ref_remote + (ps * kRows + r) * 4, __float_as_uint(o_scale), bar);
          if (lane == 0) st_async_b32(flag_remote + (ps * 4 + (warp & 3)) * 4, rose_mask, bar);
          l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        }
        if (!ok) break;
        if (!mbar_wait_warp<true, true>(smem_u32(&ctrl->ml_empty), (un & 1) ^ 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitMlEmpty;
          break;
        }
        if constexpr (kCg == 2) {
          // straight into the staging of the two O warps that store the row:
          // an arrival that releases local stores would wait for P's as well
          const uint32_t dst = p_remote + C::kStageOff + (warp & 3) * C::kStage + lane * 16 + gg * 8;
          st_async_v2(dst, __float_as_uint(m_run), __float_as_uint(l), mlfull_remote);
          st_async_v2(dst + 4 * C::kStage, __float_as_uint(m_run), __float_as_uint(l), mlfull_remote);
        } else {
          float* ml = reinterpret_cast<float*>(data + C::kMlOff);
          ml[4 * r + 2 * gg] = m_run;
          ml[4 * r + 2 * gg + 1] = l;
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mlfull_remote);
        }
        ++un;
        j0 += static_cast<uint32_t>(u.p1 - u.p0);
      }
      if (!ok && lane == 0) raise_timeout<kCg>(p, ctrl, why, j);
    }
  } else {
    // =========================== O CTA ===========================
    uint8_t* vring = data + C::kVOff;
    uint8_t* raw = data + C::kRawOff;
    if (warp == 0) {
      if (lane == 0) produce_o<kF8, kCg>(p, ctrl, kF8 ? raw : vring, &tm_o, cid, pr);
    } else if (warp == 1) {
      // ---- PV: each O CTA's warp waits until page j is ready here (V and P
      // landed, O free on a unit's first page), has its rows of O rescaled
      // where a reference rose, zeroes the slots past the sequence's end; the
      // leader then waits for the other CTA and issues PV for both.
      UnitIter it;
      it.init(p, cid);
      Unit u;
      uint32_t j = 0, un = 0, nreq = 0;
      bool ok = true;
      int why = 0;
      if (lane == 0) {
        for (int k = 0; k < C::kNP; ++k) mbar_expect_tx(smem_u32(&ctrl->p_full[k]), C::kPTx);
        if (kCg == 2) mbar_expect_tx(smem_u32(&ctrl->ml_full), C::kMlTx);
      }
      __syncwarp();
      while (ok && it.next(u)) {
        for (int vp = u.p0; vp < u.p1; ++vp, ++j) {
          const int vs = static_cast<int>(j % C::kNV);
          const int ps = static_cast<int>(j % C::kNP);
          const bool first = vp == u.p0;
          {
            const uint32_t vbar = kF8 ? smem_u32(&ctrl->v_full[vs & 3]) : smem_u32(&ctrl->kv_full[vs]);
            const uint32_t pph = (j / C::kNP) & 1;
            if (!mbar_wait_all_warp(vbar, (j / C::kNV) & 1, smem_u32(&ctrl->p_full[ps]), pph,
                                    first ? smem_u32(&ctrl->o_empty) : 0u, (un & 1) ^ 1,
                                    kCg == 2 && leader ? smem_u32(&ctrl->peer_pv[ps]) : 0u, pph, abort, p.timeout_ns)) {
              ok = false;
              why = kWaitPage;
              break;
            }
          }
          // a row's reference rose: every lane reads the four flag words
          const uint4 fw = *reinterpret_cast<const uint4*>(data + C::kFlagOff + ps * 16);
          if ((fw.x | fw.y | fw.z | fw.w) != 0u) {
            if (lane == 0) {
              ctrl->resc_page = j;
              mbar_arrive(smem_u32(&ctrl->resc_req));
            }
            if (!mbar_wait_warp(smem_u32(&ctrl->resc_done), nreq & 1, abort, p.timeout_ns)) {
              ok = false;
              why = kWaitRescDone;
              break;
            }
            ++nreq;
          }
          // this phase is done: arm the slot for page j + kNP, whose bytes
          // come only after PV(j)
          if (lane == 0) mbar_expect_tx(smem_u32(&ctrl->p_full[ps]), C::kPTx);
          uint8_t* slot = vring + vs * C::kSlotV;
          // V rows that this page has from ordinary stores: a pair's leader
          // and the other CTA order them at cluster scope
          const int valid = u.k.len - real_page(u.k, vp) * kPage;
          const bool stored = kF8 || valid < kPage;
          if constexpr (!kF8) {
            if (valid < kPage) {
              const int v0 = valid > 0 ? valid : 0;
              for (int row = v0 + (lane >> 3); row < kPage; row += 4)
#pragma unroll
                for (int box = 0; box < C::kVBoxes; ++box)
                  *reinterpret_cast<uint4*>(slot + box * C::kVBox + row * 128 + (lane & 7) * 16) =
                      make_uint4(0, 0, 0, 0);
              __syncwarp();
            }
          }
          fence_proxy_async_cta();
          tc_fence_after();
          if (kCg == 2 && !leader) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              const uint32_t bar = mapa(smem_u32(&ctrl->peer_pv[ps]), kCg);
              if (stored) mbar_arrive_shared(bar);
              else mbar_arrive_remote(bar);
            }
            continue;
          }
          if (kCg == 2 && stored) mbar_acquire_shared(smem_u32(&ctrl->peer_pv[ps]), (j / C::kNP) & 1);
          const uint64_t dv = smem_desc(smem_u32(slot), C::kVBox, 1024, kSwizzle128B);
          const uint64_t dp = smem_desc(smem_u32(data + ps * C::kPBytes), C::kPLbo, C::kPSbo, kSwizzleNone);
          // MMA h: N = 256 columns, each CTA's boxes (kVBoxes / 2) h ..
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss_cg<kCg>(tmem + h * 256, dp + static_cast<uint64_t>(k * (2 * C::kPLbo >> 4)),
                             dv + static_cast<uint64_t>((h * (C::kVBoxes / 2) * C::kVBox + k * 2048) >> 4),
                             C::kIdescPV, (first && k == 0) ? 0u : 1u);
          if (!C::kVByP) mma_commit_cg<kCg>(smem_u32(kF8 ? &ctrl->v_empty[vs & 3] : &ctrl->kv_empty[vs]), kMaskO);
          mma_commit_cg<kCg>(smem_u32(&ctrl->p_empty[ps]), kMaskAll);
          if (vp == u.p1 - 1) mma_commit_cg<kCg>(smem_u32(&ctrl->o_full), kMaskO);
        }
        ++un;
      }
      if (!ok && lane == 0) raise_timeout<kCg>(p, ctrl, why, j);
      __syncwarp();
      if (leader) {
        mma_commit_cg<kCg>(smem_u32(&ctrl->drain), static_cast<uint16_t>(1u << rank));
        if (lane == 0) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(&ctrl->drain), 0) && globaltimer_ns() - t0 < p.timeout_ns) {
          }
        }
      }
      __syncwarp();
    } else if (warp >= 4) {
      // ---- lazy O rescale and epilogue: thread r of half h (warps 4-7: 0,
      // warps 8-11: 1) owns columns [256 h, 256 h + 256) of row r.  With an
      // e4m3 cache the eight warps also expand each page's codes to f16
      // (exact), into the layout that PV reads, serving rescale requests while
      // they wait for a page or a free slot.
      const int r = (warp & 3) * 32 + lane;
      constexpr int kCols = 256;
      const int c0 = ((warp - 4) >> 2) * kCols;
      const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const float* factors = reinterpret_cast<const float*>(data + C::kRefOff);
      const uint32_t ml_remote = mapa(smem_u32(data + C::kMlOff), static_cast<uint32_t>(pr));
      uint8_t* stage = data + C::kStageOff + (warp - 4) * C::kStage;
      const uint32_t mlempty_remote = mapa(smem_u32(&ctrl->ml_empty), static_cast<uint32_t>(pr));
      const int br = pr * kRows + r;
      UnitIter it;
      it.init(p, cid);
      Unit u;
      uint32_t un = 0, nreq = 0, j = 0;
      bool ok = true;
      int why = 0;
      // Waits until the phases of both barriers have completed, serving
      // rescale requests meanwhile (a pending request holds back a PV of the
      // unit, so its o_full cannot complete while one is pending).
      auto wait_serving = [&](uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1) -> bool {
        uint64_t t0 = globaltimer_ns();
        while (true) {
          const bool req = __any_sync(0xffffffffu, mbar_try_wait(smem_u32(&ctrl->resc_req), nreq & 1));
          if (!req) {
            if (__all_sync(0xffffffffu, mbar_test4(b0, p0, b1, p1, b0, p0, b1, p1))) return true;
            if (__any_sync(0xffffffffu, *abort || globaltimer_ns() - t0 > p.timeout_ns)) {
              why = kWaitOFull;
              return false;
            }
            if (!kF8) __nanosleep(32);
            continue;
          }
          const uint32_t jr = *reinterpret_cast<volatile uint32_t*>(&ctrl->resc_page);
          const float a = br < u.k.nrows ? factors[(jr % C::kNP) * kRows + r] : 1.f;
          if (!mbar_wait_warp<false, true>(smem_u32(&ctrl->p_empty[(jr - 1) % C::kNP]), ((jr - 1) / C::kNP) & 1, abort,
                                           p.timeout_ns)) {
            why = kWaitPvPrev;
            return false;
          }
          tc_fence_after();
          if (__any_sync(0xffffffffu, a != 1.f)) {
            for (int c = c0; c < c0 + kCols; c += 16) {
              uint32_t v[16];
              tmem_ld16(tmem + lane_base + c, v);
              tmem_wait_ld_tie(v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * a);
              tmem_st16(tmem + lane_base + c, v);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&ctrl->resc_done));
          ++nreq;
          t0 = globaltimer_ns();
        }
      };
      while (ok && it.next(u)) {
        if constexpr (kF8) {
          // A lane takes 16 codes (one 16-byte chunk) at a time; four lanes a
          // row, eight rows a warp, so that the two 16-byte stores of eight
          // neighbouring lanes meet all banks once.
          const int w = warp - 4, c4 = lane & 3, r8 = lane >> 2;
          for (int vp = u.p0; vp < u.p1; ++vp, ++j) {
            const int rs = static_cast<int>(j % C::kNStO), vs = static_cast<int>(j % C::kNV);
            if (!wait_serving(smem_u32(&ctrl->kv_full[rs]), (j / C::kNStO) & 1, smem_u32(&ctrl->v_empty[vs]),
                              ((j / C::kNV) & 1) ^ 1)) {
              ok = false;
              break;
            }
            const uint8_t* src = raw + rs * C::kSlotRaw;
            uint8_t* dst = vring + vs * C::kSlotV;
            const int valid = u.k.len - real_page(u.k, vp) * kPage;
            constexpr int kItems = C::kRawBoxes * 2;  // per warp: (rows 8 ro .., half box hb), four loads in flight
#pragma unroll 1
            for (int t = 0; t < kItems; t += 4) {
              uint4 v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int item = w + 8 * (t + q), ro = item & 7, hb = item >> 3, row = ro * 8 + r8;
                const int chunk = (hb & 1) * 4 + c4;  // of the raw box's row
                v[q] = make_uint4(0, 0, 0, 0);  // slots past the sequence's end may hold anything
                if (row < valid)
                  v[q] = *reinterpret_cast<const uint4*>(src + (hb >> 1) * C::kVBox + row * 128 +
                                                         ((chunk ^ (row & 7)) << 4));
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int item = w + 8 * (t + q), ro = item & 7, hb = item >> 3, row = ro * 8 + r8;
                const uint32_t in[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
                uint32_t o[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  o[2 * k] = e4m3x2_to_f16x2(__byte_perm(in[k], 0u, 0x4140));
                  o[2 * k + 1] = e4m3x2_to_f16x2(__byte_perm(in[k], 0u, 0x4342));
                }
                uint8_t* d = dst + hb * C::kVBox + row * 128;  // half a raw box = one box of 64 values
                *reinterpret_cast<uint4*>(d + (((2 * c4) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(d + (((2 * c4 + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
              }
            }
            fence_proxy_async_cta();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(smem_u32(&ctrl->kv_empty[rs]));
              mbar_arrive(smem_u32(&ctrl->v_full[vs]));
            }
          }
          if (!ok) break;
        }
        const uint32_t of = smem_u32(&ctrl->o_full), mf = smem_u32(&ctrl->ml_full);
        if (!wait_serving(of, un & 1, of, un & 1)) {
          ok = false;
          break;
        }
        if (!mbar_wait_warp<true, true>(mf, un & 1, abort, p.timeout_ns)) {
          ok = false;
          why = kWaitMlFull;
          break;
        }
        tc_fence_after();
        float m0, l0, m1, l1;
        if constexpr (kCg == 2) {
          const float4 ml = *reinterpret_cast<const float4*>(stage + lane * 16);
          m0 = ml.x; l0 = ml.y; m1 = ml.z; l1 = ml.w;
          if (warp == 4 && lane == 0) mbar_expect_tx(mf, C::kMlTx);  // before the S CTA may send the next unit's
        } else {
          m0 = __uint_as_float(ld_cluster_u32(ml_remote + 16 * r));
          l0 = __uint_as_float(ld_cluster_u32(ml_remote + 16 * r + 4));
          m1 = __uint_as_float(ld_cluster_u32(ml_remote + 16 * r + 8));
          l1 = __uint_as_float(ld_cluster_u32(ml_remote + 16 * r + 12));
        }
        const float m_log2 = fmaxf(m0, m1);
        const float l = l0 * ex2_approx(m0 - m_log2) + l1 * ex2_approx(m1 - m_log2);
        __syncwarp();
        const int br0 = br - lane;  // the warp's first row
        bool staged = false;
        if constexpr (C::kStage > 0) staged = u.slot >= 0 ? u.slot < 2 * p.C : br0 + 32 <= u.k.nrows;
        if (!staged && lane == 0) mbar_arrive_cluster(mlempty_remote);
        const float f = store_lse<kF8>(p, u, br, c0 == 0, m_log2, l);
        if (staged) {
          store_staged<kF8, kCg>(p, u, br0, c0, tmem + lane_base, f, stage, u.slot < 0 ? &tm_out : &tm_part);
        } else {
          store_row<kF8, kCg>(p, u, br, c0, c0 + kCols, tmem + lane_base, f);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&ctrl->o_empty));
          if (staged) {  // the S CTA's sums of the next unit come into the staging
            bulk_wait_read<0>();
            mbar_arrive_cluster(mlempty_remote);
          }
        }
        ++un;
      }
      if (!ok && lane == 0) raise_timeout<kCg>(p, ctrl, why, j);
      if (lane == 0 && C::kStage > 0) bulk_wait_all();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the leaders' MMAs that read the other CTAs' memory are done
  tc_fence_after();
  if (warp == 2) tmem_dealloc_cg<kCg>(tmem, 512);
  cluster_sync();
}

// ----------------------------------------------------------------- combine
// Merges the partials of every block that slice boundaries cut (the schedule's
// list).  kParts warps share a row, each 512 / kParts of its columns: a call
// with few cut blocks gets more warps, each with more partial rows in flight.
// Lane l holds the log-sum-exps of the pieces of clusters c + l, c + l + 32,
// c + l + 64, then the warp walks the pieces in order, so that results never
// depend on timing.  The list is the schedule's, complete before the attention
// kernel began, so it is read before waiting for the latter.
constexpr int kCombineWarps = 4;

template <int kParts>
__global__ void __launch_bounds__(kCombineWarps * 32) mla_chunk_combine_kernel(const __grid_constant__ Params p) {
  constexpr int kV = 4 / kParts;      // float4s of a row per lane
  constexpr int kFly = 2 * kParts;    // partial rows in flight
  griddep_launch_dependents();
  const bool block0 = blockIdx.x == 0 && blockIdx.y == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int item = blockIdx.y * kCombineWarps + warp, br = item / kParts, col = (item % kParts) * 32 * kV + lane;
  // an earlier call's list may sit in this SM's L1: read through L2
  const bool any = static_cast<int>(blockIdx.x) < __ldcg(p.cuts);
  int4 a = make_int4(0, 0, 0, 0), b = a;
  if (any) {
    const int4* src = reinterpret_cast<const int4*>(p.cuts + 8 * (1 + static_cast<int>(blockIdx.x)));
    a = __ldcg(src);
    b = __ldcg(src + 1);
  }
  if (!any || br >= b.y) {
    if (block0) griddep_wait();  // so that this grid completes after every earlier kernel of the call
    return;
  }
  int slot[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const int cc = a.y + 32 * q + lane;
    slot[q] = -1;
    if (cc <= a.z) {
      const int4 ci = __ldcg(reinterpret_cast<const int4*>(p.cinfo + 4 * cc));
      if (ci.x < ci.y) slot[q] = cc == a.y ? a.w : 2 * cc;  // an empty slice holds no piece
    }
  }
  griddep_wait();
  float ls[3];
  float mx = -INFINITY;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    ls[q] = slot[q] >= 0 ? p.lse_part[static_cast<int64_t>(slot[q]) * p.BR + br] : -INFINITY;
    mx = ls[q] > mx || ls[q] != ls[q] ? ls[q] : mx;  // a NaN stays
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, mx, o);
    mx = (y > mx || y != y) ? y : mx;
  }
  const float base = mx == -INFINITY ? 0.f : mx;
  float w[3], z = 0.f;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    w[q] = slot[q] >= 0 ? ex2_approx((ls[q] - base) * kLog2e) : 0.f;
    z += w[q];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float inv = z == 0.f ? 0.f : 1.f / z;
  float4 acc[kV];
#pragma unroll
  for (int q = 0; q < kV; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    unsigned have = __ballot_sync(0xffffffffu, slot[q] >= 0);
    while (have) {
      float wf[kFly];
      float4 v[kFly][kV];
#pragma unroll
      for (int f = 0; f < kFly; ++f) {
        wf[f] = 0.f;
        if (have == 0) continue;
        const int src = __ffs(have) - 1;
        have &= have - 1;
        wf[f] = __shfl_sync(0xffffffffu, w[q], src) * inv;
        const int sl = __shfl_sync(0xffffffffu, slot[q], src);
        const float4* o = reinterpret_cast<const float4*>(p.o_part + (static_cast<int64_t>(sl) * p.BR + br) * kDL);
#pragma unroll
        for (int g = 0; g < kV; ++g) v[f][g] = o[col + 32 * g];
      }
#pragma unroll
      for (int f = 0; f < kFly; ++f) {
        if (wf[f] == 0.f) continue;
#pragma unroll
        for (int g = 0; g < kV; ++g) {
          acc[g].x += wf[f] * v[f][g].x; acc[g].y += wf[f] * v[f][g].y;
          acc[g].z += wf[f] * v[f][g].z; acc[g].w += wf[f] * v[f][g].w;
        }
      }
    }
  }
  const int64_t orow = static_cast<int64_t>(b.x) + br;
  uint2* dst = reinterpret_cast<uint2*>(p.out + orow * kDL * 2);
#pragma unroll
  for (int g = 0; g < kV; ++g) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[g].x, acc[g].y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[g].z, acc[g].w);
    dst[col + 32 * g] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
  if (item % kParts == 0 && lane == 0) p.lse[orow] = z == 0.f ? -INFINITY : base + __logf(z);
}

}  // namespace chunk
}  // namespace mla

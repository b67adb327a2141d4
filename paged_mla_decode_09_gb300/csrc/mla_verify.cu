// mla_verify (see include/mla_verify.h): which drafted tokens the target's
// probabilities accept, and the token that follows.
//
// A cluster of eight blocks takes a request.  Every block walks the tree by
// itself (a warp, from the nodes' entries of their parents' rows, all loaded
// at once); parents come before children, so the walk is one pass over the
// nodes.  What takes time is a pass over a whole row: the sum that a rejected
// draft leaves (z), and the last token's.  Each block adds up its part of the
// row in chunks of 256 entries, the blocks exchange their sums through
// distributed shared memory, and the block that holds the token's place finds
// the chunk by a scan of its sums and the entry by reading that chunk again.
// So a chain whose draft is rejected reads one row of each kind once: the
// sums for z are those that the token is chosen by.
//
// Sums are integers, units of 2^-60: exact in any order, so that the token is
// the one that the formula names (fp32 sums over 100K entries are off by more
// than an entry's width), without 64-bit floating point, which this chip has
// little of.
//
// What bounds it: HBM for batches (64 chains over 131072 tokens 18.0 us a call of
// a graph, 20.2 in a loop on changing inputs: 3 us until the walks end, 67 MB at
// 5-6 TB/s, 2 us for the tokens), for one request the chain of reads (offsets,
// nodes, their entries, the row, the chunk) and the barriers (32000 tokens 6.1
// in the loop).  Each rejected sibling of sampled drafts costs another pass over
// both rows, from L2, and the pass after k of them forms k - 1 products in 64 bits
// per entry, whose weight it finds anew from p and q: one request over 65536
// tokens takes 5.4 us, 7.4 with one rejected, then 17.7, 28, 52, 100, 277 and 1275
// with 2, 3, 5, 8, 16 and 40.  Fixed proposals take one pass whatever is rejected.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "mla_host.h"
#include "mla_sparse.h"
#include "mla_verify.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace verify {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 256;                       // entries that a warp adds up to one sum
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxChunks = kMaxVocab / kChunk / kCluster;  // of a block
constexpr int kNodes = MLA_TREE_MAX_NODES;
static_assert(kNodes <= kThreads && kNodes % 32 == 0, "a thread per node");

struct Params {
  const float* target;
  const float* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu_q;
  const float* accept;
  const float* sample;
  int32_t* path;
  int32_t* tokens_out;
  int32_t* num_out;
  int32_t* status;
  int64_t t_stride, d_stride;
  int32_t B, T, V, cols;
  int32_t t_vec, d_vec;  // rows are 16-byte aligned
};

// The number of [0, 1) nearest to a random number (NaN: 0).
__device__ __forceinline__ float unit(float u) { return fminf(fmaxf(u, 0.f), 0x1.fffffep-1f); }

// A value of [0, 1] in units of 2^-60, as h 2^38 + m 2^18 + l: adding a constant
// whose last place is 2^-22, 2^-42 or 2^-60 rounds to that place, and leaves the
// rounded value's integer in the sum's low bits; what was rounded off is exact.
// Integers of the bits add up in 32 bits over a few entries (the constants' own
// bits are taken off at the end).  (A conversion to 64-bit integers runs at a
// rate of two a cycle and SM: 64 rows of 131072 entries took 42 us with it.)
constexpr float kPlace1 = 2.f, kPlace2 = 0x1.8p-19f, kPlace3 = 0x1.8p-37f;
constexpr uint32_t kBits1 = 0x40000000u, kBits2 = 0x36400000u, kBits3 = 0x2d400000u;  // of these constants
struct Split {
  uint32_t h, m, l;
};
template <int kSign>
__device__ __forceinline__ void add_split(Split& s, float x) {
  const float t1 = __fadd_rn(x, kPlace1), r1 = __fsub_rn(x, __fsub_rn(t1, kPlace1));
  const float t2 = __fadd_rn(r1, kPlace2), r2 = __fsub_rn(r1, __fsub_rn(t2, kPlace2));
  const float t3 = __fadd_rn(r2, kPlace3);
  if (kSign > 0) {
    s.h += __float_as_uint(t1);
    s.m += __float_as_uint(t2);
    s.l += __float_as_uint(t3);
  } else {
    s.h -= __float_as_uint(t1);
    s.m -= __float_as_uint(t2);
    s.l -= __float_as_uint(t3);
  }
}
// the sum of what was added less what was subtracted; n: entries added less entries subtracted
__device__ __forceinline__ uint64_t joined(const Split& s, int n) {
  const int32_t h = static_cast<int32_t>(s.h - n * kBits1), m = static_cast<int32_t>(s.m - n * kBits2),
                l = static_cast<int32_t>(s.l - n * kBits3);
  return static_cast<uint64_t>((static_cast<int64_t>(h) << 38) + (static_cast<int64_t>(m) << 18) + l);
}
// A probability in units of 2^-60, rounded (NaN and below 0: 0, above 1: 1).
__device__ __forceinline__ uint64_t fixed60(float x) {
  Split s = {0u, 0u, 0u};
  add_split<1>(s, __saturatef(x));
  return joined(s, 1);
}
// a * b of such numbers, rounded down.
__device__ __forceinline__ uint64_t mul60(uint64_t a, uint64_t b) {
  return (__umul64hi(a, b) << 4) | ((a * b) >> 60);
}

struct State {
  int cur, last, cnt;  // the walk's node, the last child tested, nodes on the path
  int k;               // children rejected at cur
  int todo;            // what comes after the row's sum
  int row;             // cur's row of the probabilities; -1: a request without nodes
};
enum { kWalk = 0, kFinish = 1 };

struct Shared {
  int par[kNodes];
  int tok[kNodes];
  float acc[kNodes], wp[kNodes], wq[kNodes];  // random number, entries of the parent's rows
  int path[kNodes];
  uint64_t z[kNodes];       // draft: the sums before each rejection at cur
  int gone[kNodes];         // fixed proposals: nodes rejected at cur
  uint64_t chunk[kMaxChunks];
  uint64_t warp_sum[kWarps];
  ulonglong2 told[2][kCluster];  // every block's sum, and where its walk is
  State st;
};

// The weight of an entry after k rejections with a draft.
__device__ __forceinline__ uint64_t weight(uint64_t w, uint64_t q, const uint64_t* z, int k) {
  if (k > 0) w = w > q ? w - q : 0;  // z = 1
  for (int i = 1; i < k; ++i) {
    const uint64_t t = mul60(z[i], q);
    w = w > t ? w - t : 0;
  }
  return w;
}

__device__ __forceinline__ uint64_t warp_add(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Four entries from e on (0 behind the row's end).
__device__ __forceinline__ float4 load4(const float* row, int e, int V, bool vec) {
  if (vec && e + 4 <= V) return *reinterpret_cast<const float4*>(row + e);
  float4 v;
  v.x = e + 0 < V ? row[e + 0] : 0.f;
  v.y = e + 1 < V ? row[e + 1] : 0.f;
  v.z = e + 2 < V ? row[e + 2] : 0.f;
  v.w = e + 3 < V ? row[e + 3] : 0.f;
  return v;
}

// Whether u q < w, exactly: the product's rounding never passes w, and decides
// where it is w itself.  (Scaled, so that no product is subnormal.)
__device__ __forceinline__ bool below(float u, float q, float w) {
  const float big = q * 0x1p64f, prod = __fmul_rn(u, big), err = __fmaf_rn(u, big, -prod), lim = w * 0x1p64f;
  return prod < lim || (prod == lim && err < 0.f);
}
// Whether a b < w, all in units of 2^-60.
__device__ __forceinline__ bool below60(uint64_t a, uint64_t b, uint64_t w) {
  const uint64_t hi = __umul64hi(a, b), lim = w >> 4;
  return hi < lim || (hi == lim && a * b < w << 60);
}

// Warp 0 of a block: on from s.st to the next sum over a row.  (Every walk
// ends before one that has not been formed: a child is left to be tested where
// a walk goes on.)  `sum` is the row's sum after the last rejection (draft).
// 64-bit floating point, at about half a microsecond a test, only where a draft
// follows a rejection.
template <bool kDraft>
__device__ __forceinline__ void walk(Shared& s, int n, int q0, int cols, uint64_t sum) {
  const int lane = threadIdx.x & 31, groups = (n + 31) >> 5;
  State st = s.st;
  uint64_t z = 1ull << 60;  // fixed proposals (which end in one go)
  auto next_child = [&]() {  // of cur; -1: none
#pragma unroll 1
    for (int g = (st.last + 1) >> 5; g < groups; ++g) {
      const int i = g * 32 + lane;
      const unsigned m = __ballot_sync(0xffffffffu, i > st.last && i < n && s.par[i] == st.cur);
      if (m) return g * 32 + __ffs(m) - 1;
    }
    return -1;
  };
  st.todo = kFinish;
  while (st.cnt < cols) {
    const int j = next_child();
    if (j < 0) break;
    st.last = j;
    const float u = s.acc[j], w = __saturatef(s.wp[j]);
    bool yes;
    if (kDraft) {
      const float q = __saturatef(s.wq[j]);
      if (st.k == 0) {
        yes = below(u, q, w);
      } else {
        const double left = static_cast<double>(weight(fixed60(w), fixed60(q), s.z, st.k)) * 0x1p-60;
        yes = static_cast<double>(u) * (static_cast<double>(sum) * 0x1p-60) * static_cast<double>(q) < left;
      }
    } else {
      const int x = s.tok[j];
      bool again = false;  // a token that was rejected already has no weight left
      for (int i = lane; i < st.k; i += 32) again |= s.tok[s.gone[i]] == x;
      const uint64_t left = __any_sync(0xffffffffu, again) ? 0ull : fixed60(w);
      yes = st.k == 0 ? u < w : below60(fixed60(u), z, left);
      if (!yes) z = z > left ? z - left : 0ull;
    }
    if (yes) {
      if (lane == 0) s.path[st.cnt] = j;
      ++st.cnt;
      st.cur = j;
      st.row = q0 + j;
      st.k = 0;
      z = 1ull << 60;
      continue;
    }
    if (kDraft) {
      if (lane == 0) s.z[st.k] = st.k == 0 ? 1ull << 60 : sum;
      ++st.k;
      st.todo = next_child() < 0 ? kFinish : kWalk;
      break;
    }
    if (lane == 0) s.gone[st.k] = j;
    __syncwarp();
    ++st.k;
  }
  __syncwarp();
  if (lane == 0) s.st = st;
}

template <bool kDraft>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 4)
    mla_verify_kernel(const __grid_constant__ Params p) {
  __shared__ Shared s;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_ctarank());
  const int b = static_cast<int>(cluster_id_x());
  cluster_arrive();  // waited for before a block writes to another's shared memory
  int q0 = p.cu_q[b];
  const int q1 = p.cu_q[b + 1];
  int n = q1 - q0, flag = 0;
  if (!(q0 >= 0 && q1 >= q0 && q1 <= p.T && (b > 0 || q0 == 0))) {
    n = q0 = 0;
    flag = MLA_DEV_BAD_QUERY_RANGE;
  } else if (n > kNodes) {
    n = q0 = 0;
    flag = MLA_DEV_BAD_TREE;
  }
  int32_t* path = p.path + static_cast<int64_t>(b) * p.cols;
  int32_t* next = p.tokens_out + static_cast<int64_t>(b) * p.cols;
  if (flag && rank == 0 && tid == 0) atomicOr(p.status, flag);
  flag = 0;
  if (tid < n) {
    int par = -2, tok = 0;
    if (tid > 0) {
      par = p.parents[q0 + tid];
      tok = p.tokens[q0 + tid];
      if (par < -1 || par >= tid) {
        flag |= MLA_DEV_BAD_TREE;
        par = -2;
      }
      if (tok < 0 || tok >= p.V) {
        flag |= MLA_DEV_BAD_INDEX;
        par = -2;
      }
    } else if (p.parents[q0] != -1) {
      flag |= MLA_DEV_BAD_TREE;
    }
    s.par[tid] = par;
    s.tok[tid] = tok;
    if (par >= 0) {
      s.acc[tid] = unit(p.accept[q0 + tid]);
      s.wp[tid] = p.target[(q0 + par) * p.t_stride + tok];
      if (kDraft) s.wq[tid] = p.draft[(q0 + par) * p.d_stride + tok];
    }
    if (flag && rank == 0) atomicOr(p.status, flag);
  }
  if (rank == 0)  // (the block that finds the last token writes it later)
    for (int k = tid; k < p.cols; k += kThreads) next[k] = -1;
  if (tid == 0) {
    s.path[0] = 0;
    s.st = {0, 0, n > 0 ? 1 : 0, 0, kFinish, n > 0 ? q0 : -1};
  }
  __syncthreads();
  const int all = (p.V + kChunk - 1) / kChunk, per = (all + kCluster - 1) / kCluster;
  const int c0 = rank * per < all ? rank * per : all, chunks = (all - c0 < per ? all - c0 : per);
  uint64_t sum = 0;      // of the row's weights, all blocks
  int pass = 0;
  const float* tr = nullptr;
  const float* dr = nullptr;
  State st = {};
  auto gone = [&](int i) { return s.gone[i] & (kNodes - 1); };  // (a state taken over may count more than this block has)

  // adds up the weights of st.row after st.k rejections.  The blocks walk by
  // themselves, on the same inputs; the first one's state goes with its sum and
  // is taken over by all, so that they use the same barriers, and stay within
  // the rows, even if another stream changes the inputs meanwhile
  auto add_up = [&]() {
    const int nc = st.row < 0 ? 0 : chunks;
    tr = p.target + (st.row < 0 ? 0 : st.row) * p.t_stride;
    if (kDraft) dr = p.draft + (st.row < 0 ? 0 : st.row) * p.d_stride;
    const bool tv = p.t_vec != 0, dv = p.d_vec != 0, rest = kDraft && st.k == 1;
    constexpr int kFly = 2;  // chunks of a warp in flight
    uint64_t mine = 0;       // of this warp's chunks
    if (kDraft && st.k > 1) {  // behind rejected siblings: entry by entry
#pragma unroll 1
      for (int c = warp; c < nc; c += kWarps) {
        const int e = (c0 + c) * kChunk + lane * 4;
        const float4 a[2] = {load4(tr, e, p.V, tv), load4(tr, e + 128, p.V, tv)};
        const float4 q[2] = {load4(dr, e, p.V, dv), load4(dr, e + 128, p.V, dv)};
        uint64_t v = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v += weight(fixed60(a[h].x), fixed60(q[h].x), s.z, st.k) + weight(fixed60(a[h].y), fixed60(q[h].y), s.z, st.k);
          v += weight(fixed60(a[h].z), fixed60(q[h].z), s.z, st.k) + weight(fixed60(a[h].w), fixed60(q[h].w), s.z, st.k);
        }
        v = warp_add(v);
        if (lane == 0) s.chunk[c] = v;
        mine += v;
      }
    } else
#pragma unroll 1
    for (int c = warp; c < nc; c += kWarps * kFly) {
      float4 a[kFly][2], q[kFly][2];
#pragma unroll
      for (int f = 0; f < kFly; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int e = (c0 + c + f * kWarps) * kChunk + h * 128 + lane * 4;
          if (c + f * kWarps < nc) {
            a[f][h] = load4(tr, e, p.V, tv);
            if (rest) q[f][h] = load4(dr, e, p.V, dv);
          }
        }
#pragma unroll
      for (int f = 0; f < kFly; ++f) {
        if (c + f * kWarps >= nc) break;
        Split sp = {0u, 0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float x[4] = {a[f][h].x, a[f][h].y, a[f][h].z, a[f][h].w};
          const float y[4] = {q[f][h].x, q[f][h].y, q[f][h].z, q[f][h].w};
          if (!rest) {
#pragma unroll
            for (int e = 0; e < 4; ++e) add_split<1>(sp, __saturatef(x[e]));
          } else {  // p - q where that is above 0
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float c = __saturatef(x[e]), d = __saturatef(y[e]);
              add_split<1>(sp, c > d ? c : 0.f);
              add_split<-1>(sp, c > d ? d : 0.f);
            }
          }
        }
        const uint64_t v = warp_add(joined(sp, rest ? 0 : 8));
        if (lane == 0) s.chunk[c + f * kWarps] = v;
        mine += v;
      }
    }
    if (lane == 0) s.warp_sum[warp] = mine;
    __syncthreads();
    if (!kDraft && st.k > 0) {  // tokens that were rejected have no weight left
      if (tid < st.k) {
        const int x = s.tok[gone(tid)], c = x / kChunk - c0;
        bool first = c >= 0 && c < nc;
        for (int i = 0; first && i < tid; ++i) first = s.tok[gone(i)] != x;
        if (first) {
          const unsigned long long less = 0ull - fixed60(s.wp[gone(tid)]);
          atomicAdd(reinterpret_cast<unsigned long long*>(&s.chunk[c]), less);
          atomicAdd(reinterpret_cast<unsigned long long*>(&s.warp_sum[0]), less);
        }
      }
      __syncthreads();
    }
    if (warp == 0) {
      const uint64_t v = warp_add(lane < kWarps ? s.warp_sum[lane] : 0ull);
      if (pass == 0) cluster_wait();  // every block has begun
      if (lane < kCluster) {
        const uint32_t dst = mapa(smem_u32(&s.told[pass & 1][rank]), static_cast<uint32_t>(lane));
        // (cur, last, k and cnt - 1 are below 256; rows below 2^31 - 1, which stands for none)
        const uint32_t lo = static_cast<uint32_t>(st.cur | st.last << 8 | (st.k & 255) << 16) |
                            static_cast<uint32_t>(st.cnt - 1) << 24;
        const uint32_t hi = (st.row < 0 ? 0x7fffffffu : static_cast<uint32_t>(st.row)) |
                            static_cast<uint32_t>(st.todo) << 31;
        st_cluster_v4(dst, make_uint4(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32), lo, hi));
      }
    }
    if (pass == 0 && warp != 0) cluster_wait();
    cluster_sync();
    sum = 0;
#pragma unroll
    for (int r = 0; r < kCluster; ++r) sum += s.told[pass & 1][r].x;
    const uint32_t lo = static_cast<uint32_t>(s.told[pass & 1][0].y), hi = static_cast<uint32_t>(s.told[pass & 1][0].y >> 32);
    const bool some = (hi & 0x7fffffffu) != 0x7fffffffu;
    st.cur = static_cast<int>(lo & 255u);
    st.last = static_cast<int>(lo >> 8 & 255u);
    st.k = static_cast<int>(lo >> 16 & 255u);
    st.cnt = some ? static_cast<int>(lo >> 24) + 1 : 0;
    st.todo = static_cast<int>(hi >> 31);
    st.row = some ? static_cast<int>(hi & 0x7fffffffu) : -1;
    ++pass;
  };

  while (true) {
    if (warp == 0) walk<kDraft>(s, n, q0, p.cols, sum);
    __syncthreads();
    st = s.st;
    add_up();
    if (st.todo == kFinish) break;
    if (tid == 0) s.st = st;
    __syncwarp();
  }
  if (sum == 0 && st.row >= 0) {  // rounding has left nothing: the node's own row
    st.k = 0;
    add_up();
  }
  if (warp > 0) {  // the outputs but the last token
    if (rank != 0) return;
    for (int k = tid - 32; k < p.cols; k += kThreads - 32) {
      path[k] = k < st.cnt ? s.path[k] : -1;
      if (k < st.cnt - 1) next[k] = s.tok[s.path[k + 1]];
    }
    if (tid == 32) {
      p.num_out[b] = st.cnt;
      if (sum == 0 && st.row >= 0) atomicOr(p.status, MLA_DEV_BAD_PROBS);
    }
    return;
  }
  if (sum == 0) return;
  const float u = unit(p.sample[b]);
  uint64_t at = mul60(fixed60(u), sum);  // below sum
  const int last_pass = (pass - 1) & 1;
  bool here = true;
#pragma unroll
  for (int r = 0; r < kCluster; ++r)
    if (r < rank) {
      here = here && at >= s.told[last_pass][r].x;
      at -= s.told[last_pass][r].x;
    }
  if (!here || at >= s.told[last_pass][rank].x) return;
  // the chunk: each lane some, in order
  const int each = (chunks + 31) / 32, first = lane * each;
  uint64_t mine = 0, before;
#pragma unroll 1
  for (int c = first; c < first + each && c < chunks; ++c) mine += s.chunk[c];
  before = warp_scan(mine) - mine;
  const unsigned who = __ballot_sync(0xffffffffu, at >= before && at - before < mine);
  if (who == 0) return;
  int pick = first;
  uint64_t left = at - before;
  if (lane == __ffs(who) - 1)
    while (left >= s.chunk[pick]) left -= s.chunk[pick++];
  pick = c0 + __shfl_sync(0xffffffffu, pick, __ffs(who) - 1);
  at = __shfl_sync(0xffffffffu, left, __ffs(who) - 1);
  // the entry: each lane eight, in order
  uint64_t w[kChunk / 32];
  mine = 0;
  const int e0 = pick * kChunk + lane * (kChunk / 32);
  static_assert(kChunk == 256, "two quads a lane");
  const float4 a0 = load4(tr, e0, p.V, p.t_vec), a1 = load4(tr, e0 + 4, p.V, p.t_vec);
  const float a[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
  float4 d0 = make_float4(0.f, 0.f, 0.f, 0.f), d1 = d0;
  if (kDraft && st.k > 0) {
    d0 = load4(dr, e0, p.V, p.d_vec);
    d1 = load4(dr, e0 + 4, p.V, p.d_vec);
  }
  const float d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
#pragma unroll
  for (int e = 0; e < kChunk / 32; ++e) {
    w[e] = fixed60(a[e]);
    if (kDraft) {
      if (st.k > 0) w[e] = weight(w[e], fixed60(d[e]), s.z, st.k);
    } else {
      for (int i = 0; i < st.k; ++i)
        if (s.tok[gone(i)] == e0 + e) w[e] = 0;
    }
    mine += w[e];
  }
  before = warp_scan(mine) - mine;
  if (at >= before && at - before < mine) {
    int y = e0;
#pragma unroll
    for (int e = 0; e < kChunk / 32; ++e) {
      if (at >= before) y = e0 + e;
      before += w[e];
    }
    next[st.cnt - 1] = y;
  }
}

}  // namespace verify
}  // namespace mla

extern "C" int mla_verify(const mla_verify_dims* d, const float* target, const float* draft, const int32_t* tokens,
                          const int32_t* parents, const int32_t* cu_q_lens, const float* accept, const float* sample,
                          int32_t* path, int32_t* tokens_out, int32_t* num_out, int32_t* status, void* stream) {
  using mla::host::aligned;
  if (!d || !target || !tokens || !parents || !cu_q_lens || !accept || !sample || !path || !tokens_out || !num_out ||
      !status)
    return MLA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->total_q < 1 || d->vocab < 1 || d->path_cols < 1 || d->target_stride < d->vocab ||
      (draft && d->draft_stride < d->vocab))
    return MLA_ERR_INVALID_ARG;
  if (d->batch > 1 << 27 || d->vocab > mla::verify::kMaxVocab || d->target_stride > (1ll << 40) ||
      (draft && d->draft_stride > (1ll << 40)))
    return MLA_ERR_UNSUPPORTED;
  // every block of a request reads its inputs, one writes the outputs
  {
    const int64_t T = d->total_q, B = d->batch, cells = B * d->path_cols;
    const struct {
      const void* at;
      int64_t bytes;
    } outs[] = {{path, 4 * cells}, {tokens_out, 4 * cells}, {num_out, 4 * B}, {status, 4}},
      ins[] = {{tokens, 4 * T}, {parents, 4 * T}, {cu_q_lens, 4 * B + 4}, {accept, 4 * T}, {sample, 4 * B}};
    for (int i = 0; i < 4; ++i) {
      for (int j = 0; j < i; ++j)
        if (mla::host::overlap(outs[i].at, outs[i].bytes, outs[j].at, outs[j].bytes)) return MLA_ERR_INVALID_ARG;
      for (const auto& in : ins)
        if (mla::host::overlap(outs[i].at, outs[i].bytes, in.at, in.bytes)) return MLA_ERR_INVALID_ARG;
      const int64_t words = outs[i].bytes / 4;
      if (mla::host::overlap_rows(target, T, d->target_stride, d->vocab, outs[i].at, words) ||
          (draft && mla::host::overlap_rows(draft, T, d->draft_stride, d->vocab, outs[i].at, words)))
        return MLA_ERR_INVALID_ARG;
    }
  }
  if (!aligned(target, 4) || !aligned(draft, 4) || !aligned(tokens, 4) || !aligned(parents, 4) ||
      !aligned(cu_q_lens, 4) || !aligned(accept, 4) || !aligned(sample, 4) || !aligned(path, 4) ||
      !aligned(tokens_out, 4) || !aligned(num_out, 4) || !aligned(status, 4))
    return MLA_ERR_ALIGNMENT;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  const int rc = mla::host::device_ok(dev);
  if (rc != MLA_OK) return rc;
  using namespace mla::verify;
  Params p;
  p.target = target;
  p.draft = draft;
  p.tokens = tokens;
  p.parents = parents;
  p.cu_q = cu_q_lens;
  p.accept = accept;
  p.sample = sample;
  p.path = path;
  p.tokens_out = tokens_out;
  p.num_out = num_out;
  p.status = status;
  p.t_stride = d->target_stride;
  p.d_stride = draft ? d->draft_stride : 0;
  p.B = d->batch;
  p.T = d->total_q;
  p.V = d->vocab;
  p.cols = d->path_cols;
  p.t_vec = aligned(target, 16) && p.t_stride % 4 == 0;
  p.d_vec = draft && aligned(draft, 16) && p.d_stride % 4 == 0;
  const dim3 grid(static_cast<unsigned>(p.B) * kCluster), block(kThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = draft ? mla::host::launch_pdl(&mla_verify_kernel<true>, grid, block, 0, s, 0, p)
                              : mla::host::launch_pdl(&mla_verify_kernel<false>, grid, block, 0, s, 0, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

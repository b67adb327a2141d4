// mla_rope_pack (see include/mla_rope.h): a step's query and key parts rotated,
// its rows written into the paged cache.
//
// Angles: a frequency is a 64-bit fraction F of a turn, so position * F modulo
// 2^64 is the angle's fraction of a turn, with no range reduction and no loss at
// far positions; as a signed number it is the angle in half turns, [-1, 1), for
// sincospi in fp32 (2^-25 of a half turn from its conversion).  R / 2 of them a
// token, once for all heads.
//
// Work: a block takes a few tokens.  A head's 64 values are four items of two
// 16-byte chunks, chosen so that an item needs the same eight angles in both
// layouts (interleaved: chunks 2 i and 2 i + 1; halves: chunk i and the one
// R / 2 behind it); a thread's items are all of one i.  The loads of queries and rows do not depend on the request: they
// are in flight while the block looks its tokens up (offsets, length, page:
// three dependent reads) and forms the angles.
//
// What bounds it: HBM for prompts (each query value read and written once, each
// row read and written once: 6.1K tokens of 128 heads into an e4m3 cache 36 us,
// 5.5 TB/s of the 6.8 that a copy reaches), the chain of dependent reads for a
// few tokens (4 tokens of 16 heads 3.2 us a call of a graph).  Swept: two items in flight and five
// blocks an SM; three and five 38.2 us, three and four 35.3 (64 trees of 16
// tokens 7.5 us instead of 6.7), two and six 37.5; streaming hints 36.3-36.5.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "mla_e4m3.cuh"
#include "mla_host.h"
#include "mla_rope.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace rope {

constexpr int kPage = 64;
constexpr int kRowVals = 576;
constexpr int kLatChunks = 64;   // 16-byte chunks of c_kv
constexpr int kThreads = 256;
constexpr int kMaxTok = 16;      // tokens of a block
constexpr int kAhead = 2;        // items and chunks a thread has in flight

struct Params {
  const uint8_t* q_pe;
  const uint8_t* rows;
  const int32_t* positions;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;
  uint8_t* q_out;
  uint8_t* cache;
  int32_t* status;
  int64_t q_tok, q_head, row;  // strides in bytes
  int32_t B, H, T, num_pages, max_pages, pt_stride, R, toks, more;
  float amp;
  e4m3::Scale sc;
  uint64_t turn[32];
};

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The two chunks of item i of a head: rotating items first, then those that pass.
__device__ __forceinline__ void chunks_of(int i, int R, bool inter, int& c0, int& c1) {
  const bool halves = !inter && i < (R >> 4);
  c0 = halves ? i : 2 * i;
  c1 = halves ? i + (R >> 4) : 2 * i + 1;
}

// Rotates an item's two chunks by its eight angles (cosines, then sines).
template <bool kInter>
__device__ __forceinline__ void turn8(float (&a)[8], float (&b)[8], const float (&cs)[16]) {
  float co[8], si[8];
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const float4 c = *reinterpret_cast<const float4*>(cs + k), s = *reinterpret_cast<const float4*>(cs + 8 + k);
    co[k] = c.x; co[k + 1] = c.y; co[k + 2] = c.z; co[k + 3] = c.w;
    si[k] = s.x; si[k + 1] = s.y; si[k + 2] = s.z; si[k + 3] = s.w;
  }
  if constexpr (kInter) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a0 = a[2 * k], a1 = a[2 * k + 1], b0 = b[2 * k], b1 = b[2 * k + 1];
      a[2 * k] = a0 * co[k] - a1 * si[k];
      a[2 * k + 1] = a0 * si[k] + a1 * co[k];
      b[2 * k] = b0 * co[4 + k] - b1 * si[4 + k];
      b[2 * k + 1] = b0 * si[4 + k] + b1 * co[4 + k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = a[k], y = b[k];
      a[k] = x * co[k] - y * si[k];
      b[k] = x * si[k] + y * co[k];
    }
  }
}

template <bool kF8, bool kInter>
__global__ void __launch_bounds__(kThreads, 5) mla_rope_pack_kernel(const __grid_constant__ Params p) {
  __shared__ int s_req[kMaxTok];
  __shared__ int64_t s_slot[kMaxTok];                        // cache row, -1: not written
  __shared__ __align__(16) float s_cs[kMaxTok][4][16];       // per item: eight cosines, eight sines
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  // the tokens in equal parts (the first p.more blocks take one more)
  const int bx = static_cast<int>(blockIdx.x), nt = p.toks + (bx < p.more ? 1 : 0);
  const int t0 = bx * p.toks + (bx < p.more ? bx : p.more);
  const int per = p.H * 4;                      // query items of a token
  const int items = nt * per, lats = nt * kLatChunks;
  // first loads: query items tid, tid + 256, ..; c_kv chunks likewise
  auto q_at = [&](int it, int& c0, int& c1) -> const uint8_t* {
    const int k = it / per, r = it - k * per;
    chunks_of(r & 3, p.R, kInter, c0, c1);
    return p.q_pe + (t0 + k) * p.q_tok + (r >> 2) * p.q_head;
  };
  uint4 qa[kAhead], qb[kAhead], lat[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int it = tid + u * kThreads;
    if (it < items) {
      int c0, c1;
      const uint8_t* src = q_at(it, c0, c1);
      qa[u] = ldg16(src + 16 * c0);
      qb[u] = ldg16(src + 16 * c1);
    }
    if (it < lats) lat[u] = ldg16(p.rows + (t0 + (it >> 6)) * p.row + 16 * (it & 63));
  }
  // each token's request
  if (tid < kMaxTok) s_req[tid] = -1;
  __syncthreads();
  for (int b = tid; b < p.B; b += kThreads) {
    const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > p.T || (b == 0 && q0 != 0)) {
      if (blockIdx.x == 0) atomicOr(p.status, MLA_DEV_BAD_QUERY_RANGE);
      continue;
    }
    const int lo = q0 > t0 ? q0 : t0, hi = q1 < t0 + nt ? q1 : t0 + nt;
    for (int t = lo; t < hi; ++t) atomicMax(&s_req[t - t0], b);  // (offsets that decrease: the last that names it)
  }
  __syncthreads();
  // its slot, and its angles
  int fail = 0, mine = -1;
  if (tid < nt) {
    const int b = s_req[tid];
    int64_t slot = -1;
    if (b >= 0) {
      const int q0 = p.cu_q[b], n = p.cu_q[b + 1] - q0, L = p.seq_lens[b];
      if (L < n || L > p.max_pages * kPage) {
        fail = MLA_DEV_BAD_SEQ_LEN;
        mine = tid;
      } else {
        const int at = L - n + (t0 + tid - q0);  // (in the table, unless offsets change under the call)
        const bool in = at >= 0 && at < p.max_pages * kPage;
        const int page = in ? p.page_table[static_cast<int64_t>(b) * p.pt_stride + at / kPage] : -1;
        if (page < 0 || page >= p.num_pages) fail = MLA_DEV_BAD_PAGE_ID;
        else slot = static_cast<int64_t>(page) * kPage + at % kPage;
      }
    }
    s_slot[tid] = slot;
  }
  const int half = p.R >> 1;
  for (int x = tid; x < nt * 32; x += kThreads) {
    const int k = x >> 5, i = x & 31, b = s_req[k];
    if (i >= half || b < 0) continue;
    int pos;
    if (p.positions) pos = p.positions[t0 + k];
    else pos = p.seq_lens[b] - p.cu_q[b + 1] + t0 + k;  // (used only if the length is right)
    const int64_t phase = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.turn[i]);
    float si, co;
    sincospif(static_cast<float>(phase) * 0x1p-63f, &si, &co);
    s_cs[k][i >> 3][i & 7] = co * p.amp;
    s_cs[k][i >> 3][8 + (i & 7)] = si * p.amp;
  }
  if (fail != 0) atomicOr(p.status, fail);
  __syncthreads();
  if (mine >= 0) s_req[mine] = -1;  // a bad length: left out
  __syncthreads();

  // queries: a thread's items are all of one number i when 256 is a multiple of 4
  const int i = tid & 3;
  const bool turns = i < (p.R >> 4);
  auto put_q = [&](int it, const uint4& va, const uint4& vb) {
    const int k = it / per, r = it - k * per;
    if (s_req[k] < 0) return;
    int c0, c1;
    chunks_of(i, p.R, kInter, c0, c1);
    uint8_t* dst = p.q_out + (static_cast<int64_t>(t0 + k) * p.H + (r >> 2)) * 128;
    if (!turns) {
      *reinterpret_cast<uint4*>(dst + 16 * c0) = va;
      *reinterpret_cast<uint4*>(dst + 16 * c1) = vb;
      return;
    }
    float a[8], b[8];
    unpack(va, a);
    unpack(vb, b);
    turn8<kInter>(a, b, s_cs[k][i]);
    *reinterpret_cast<uint4*>(dst + 16 * c0) = pack(a);
    *reinterpret_cast<uint4*>(dst + 16 * c1) = pack(b);
  };
  auto put_lat = [&](int it, const uint4& v) {
    const int64_t slot = s_slot[it >> 6];
    if (slot < 0) return;
    if constexpr (kF8) reinterpret_cast<uint2*>(p.cache + slot * kRowVals)[it & 63] = e4m3::e4m3x8(v, p.sc);
    else reinterpret_cast<uint4*>(p.cache + slot * kRowVals * 2)[it & 63] = v;
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int it = tid + u * kThreads;
    if (it < items) put_q(it, qa[u], qb[u]);
    if (it < lats) put_lat(it, lat[u]);
  }
  for (int base = kAhead * kThreads; base < items; base += kAhead * kThreads) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int it = base + tid + u * kThreads;
      if (it >= items) continue;
      int c0, c1;
      const uint8_t* src = q_at(it, c0, c1);
      qa[u] = ldg16(src + 16 * c0);
      qb[u] = ldg16(src + 16 * c1);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int it = base + tid + u * kThreads;
      if (it < items) put_q(it, qa[u], qb[u]);
    }
  }
  for (int it = kAhead * kThreads + tid; it < lats; it += kThreads)
    put_lat(it, ldg16(p.rows + (t0 + (it >> 6)) * p.row + 16 * (it & 63)));
  // k_pe of each token: four items
  for (int it = tid; it < nt * 4; it += kThreads) {
    const int k = it >> 2;
    const int64_t slot = s_slot[k];
    if (slot < 0) continue;
    int c0, c1;
    chunks_of(i, p.R, kInter, c0, c1);
    const uint8_t* src = p.rows + (t0 + k) * p.row + 1024;
    const uint4 va = ldg16(src + 16 * c0), vb = ldg16(src + 16 * c1);
    float a[8], b[8];
    unpack(va, a);
    unpack(vb, b);
    if (turns) turn8<kInter>(a, b, s_cs[k][i]);
    if constexpr (kF8) {
      uint2* dst = reinterpret_cast<uint2*>(p.cache + slot * kRowVals + 512);
      dst[c0] = e4m3::e4m3x8(a, p.sc);
      dst[c1] = e4m3::e4m3x8(b, p.sc);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(p.cache + slot * kRowVals * 2 + 1024);
      dst[c0] = turns ? pack(a) : va;
      dst[c1] = turns ? pack(b) : vb;
    }
  }
}

}  // namespace rope
}  // namespace mla

namespace {

using mla::host::aligned;
using mla::host::overlap;
using mla::host::overlap_rows;

bool rotary_ok(int32_t r) { return r >= 16 && r <= 64 && r % 16 == 0; }

constexpr double kTwoPi = 6.283185307179586476925;

// What both frequency functions refuse.
int frequencies_ok(int32_t rotary_dim, double base, double factor, int32_t original_len, double fast, double slow,
                   const double* out) {
  if (!out || !std::isfinite(base) || base < 1.0 || !std::isfinite(factor) || factor < 1.0 || original_len < 0)
    return MLA_ERR_INVALID_ARG;
  if (original_len > 0 && (!std::isfinite(fast) || !std::isfinite(slow) || fast <= slow)) return MLA_ERR_INVALID_ARG;
  return rotary_ok(rotary_dim) ? MLA_OK : MLA_ERR_UNSUPPORTED;
}

// A frequency of which a share `keep`, limited to [0, 1], stays and the rest is divided by the factor.
double scaled(double f, double factor, double keep) {
  const double g = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
  return factor == 1.0 ? f : g * f + (1.0 - g) * f / factor;
}

}  // namespace

extern "C" {

int mla_rope_frequencies(int32_t rotary_dim, double base, double factor, int32_t original_len, double fast,
                         double slow, double* out) {
  const int rc = frequencies_ok(rotary_dim, base, factor, original_len, fast, slow, out);
  if (rc != MLA_OK) return rc;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rotary_dim);
    out[i] = scaled(f, factor, original_len > 0 ? (original_len * f / kTwoPi - slow) / (fast - slow) : 0.0);
  }
  return MLA_OK;
}

int mla_rope_frequencies_by_index(int32_t rotary_dim, double base, double factor, int32_t original_len, double fast,
                                  double slow, double* out) {
  const int rc = frequencies_ok(rotary_dim, base, factor, original_len, fast, slow, out);
  if (rc != MLA_OK) return rc;
  double lo = 0.0, hi = 0.0;
  if (original_len > 0) {
    if (base <= 1.0 || slow <= 0.0) return MLA_ERR_INVALID_ARG;
    auto index_of = [&](double turns) {
      return rotary_dim * std::log(original_len / (kTwoPi * turns)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(index_of(fast)), 0.0);
    hi = std::fmin(std::ceil(index_of(slow)), rotary_dim - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double keep = 0.0;
    if (original_len > 0) keep = hi > lo ? 1.0 - (i - lo) / (hi - lo) : (i <= lo ? 1.0 : 0.0);
    out[i] = scaled(std::pow(base, -2.0 * i / rotary_dim), factor, keep);
  }
  return MLA_OK;
}

int mla_rope_plan_init(int32_t rotary_dim, int32_t interleaved, float amplitude, const double* frequencies,
                       mla_rope_plan* plan) {
  if (!frequencies || !plan || !std::isfinite(amplitude) || amplitude <= 0.f) return MLA_ERR_INVALID_ARG;
  if (!rotary_ok(rotary_dim)) return MLA_ERR_UNSUPPORTED;
  mla_rope_plan r = {};
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = frequencies[i];
    if (!(f >= 0.0) || f >= kTwoPi) return MLA_ERR_INVALID_ARG;
    const double t = f / kTwoPi;  // < 1; a quotient that rounds to 1 is no turn at all
    r.turn[i] = t < 1.0 ? static_cast<uint64_t>(t * 0x1p64) : 0;
  }
  r.rotary_dim = rotary_dim;
  r.interleaved = interleaved != 0;
  r.amplitude = amplitude;
  *plan = r;
  return MLA_OK;
}

int mla_rope_pack(const mla_rope_dims* d, const mla_rope_plan* plan, const void* q_pe, const void* rows,
                  const int32_t* positions, const int32_t* page_table, const int32_t* seq_lens,
                  const int32_t* cu_q_lens, float kv_scale, void* q_out, void* kv_cache, int32_t* status,
                  void* stream_v) {
  if (!d || !plan || !q_pe || !rows || !page_table || !seq_lens || !cu_q_lens || !q_out || !kv_cache || !status)
    return MLA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_heads < 1 || d->total_q < 1 || d->num_pages < 1 || d->max_pages_per_req < 1 ||
      d->page_table_stride < d->max_pages_per_req)
    return MLA_ERR_INVALID_ARG;
  const int64_t T = d->total_q, H = d->num_heads;
  const int64_t q_head = H > 1 ? d->q_head_stride : 64, q_tok = T > 1 ? d->q_token_stride : 64;
  const int64_t row = T > 1 ? d->row_stride : 576;
  if (q_head < 64 || q_tok < 64 || row < 576) return MLA_ERR_INVALID_ARG;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  if (!rotary_ok(plan->rotary_dim) || H > 65536 || T * H > INT_MAX || static_cast<int64_t>(d->max_pages_per_req) * 64 > INT_MAX ||
      q_head > (1ll << 40) || q_tok > (1ll << 40) || row > (1ll << 40))
    return MLA_ERR_UNSUPPORTED;
  if (!std::isfinite(plan->amplitude) || plan->amplitude <= 0.f) return MLA_ERR_INVALID_ARG;
  const bool f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  if (f8 && !mla::e4m3::scale_ok(kv_scale)) return MLA_ERR_INVALID_ARG;
  {  // blocks look up their tokens, and read their rows, after others have written
    const int64_t B = d->batch, words = T * H * 32;  // of q_out
    const struct {
      const int32_t* at;
      int64_t n;
    } ins[] = {{positions, T}, {seq_lens, B}, {cu_q_lens, B + 1}};
    for (const auto& in : ins)
      if (in.at && (overlap(q_out, 4 * words, in.at, 4 * in.n) || overlap(status, 4, in.at, 4 * in.n)))
        return MLA_ERR_INVALID_ARG;
    if (overlap_rows(page_table, B, d->page_table_stride, d->max_pages_per_req, q_out, words) ||
        overlap_rows(page_table, B, d->page_table_stride, d->max_pages_per_req, status, 1) ||
        overlap_rows(rows, T, row / 2, 288, q_out, words) || overlap_rows(rows, T, row / 2, 288, status, 1) ||
        overlap(q_out, 4 * words, status, 4))
      return MLA_ERR_INVALID_ARG;
  }
  if (!aligned(q_pe, 16) || !aligned(rows, 16) || !aligned(q_out, 16) || !aligned(kv_cache, 16) || q_head % 8 != 0 ||
      q_tok % 8 != 0 || row % 8 != 0 || !aligned(positions, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_q_lens, 4) || !aligned(status, 4))
    return MLA_ERR_ALIGNMENT;
  const bool same = q_pe == q_out && (H == 1 || q_head == 64) && (T == 1 || q_tok == H * 64);
  if (!same && overlap(q_pe, 2 * ((T - 1) * q_tok + (H - 1) * q_head + 64), q_out, T * H * 128))
    return MLA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  const int rc = mla::host::device_ok(dev);
  if (rc != MLA_OK) return rc;
  using namespace mla::rope;
  Params p;
  p.q_pe = static_cast<const uint8_t*>(q_pe);
  p.rows = static_cast<const uint8_t*>(rows);
  p.positions = positions;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q_lens;
  p.q_out = static_cast<uint8_t*>(q_out);
  p.cache = static_cast<uint8_t*>(kv_cache);
  p.status = status;
  p.q_tok = 2 * q_tok;
  p.q_head = 2 * q_head;
  p.row = 2 * row;
  p.B = d->batch;
  p.H = d->num_heads;
  p.T = d->total_q;
  p.num_pages = d->num_pages;
  p.max_pages = d->max_pages_per_req;
  p.pt_stride = d->page_table_stride;
  p.R = plan->rotary_dim;
  p.amp = plan->amplitude;
  p.sc = mla::e4m3::scale_of(f8 ? kv_scale : 1.0f);
  for (int i = 0; i < 32; ++i) p.turn[i] = i < p.R / 2 ? plan->turn[i] : 0;
  // blocks: their tokens give each thread an item or two, but there is one for
  // every SM first; where more would run than fit at once, whole rounds of them
  // with about eight tokens each, whose look-ups are one chain (6K tokens of 128
  // heads: 45 us at a token a block, 36 at eight, 45 in one round and a third)
  constexpr int64_t kAtOnce = 152 * 5;
  int64_t toks = (kAhead * kThreads) / (4 * H);
  toks = toks < 1 ? 1 : (toks > kMaxTok - 1 ? kMaxTok - 1 : toks);
  const int64_t spread = (T + 151) / 152, most = toks > 9 ? toks : 9;
  toks = toks < spread ? toks : spread;
  int64_t blocks = (T + toks - 1) / toks;
  if (blocks > kAtOnce) blocks = kAtOnce * ((T + kAtOnce * most - 1) / (kAtOnce * most));
  p.toks = static_cast<int32_t>(T / blocks);
  p.more = static_cast<int32_t>(T % blocks);
  const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
  cudaStream_t s = static_cast<cudaStream_t>(stream_v);
  const bool inter = plan->interleaved != 0;
  auto* kernel = f8 ? (inter ? &mla_rope_pack_kernel<true, true> : &mla_rope_pack_kernel<true, false>)
                    : (inter ? &mla_rope_pack_kernel<false, true> : &mla_rope_pack_kernel<false, false>);
  if (mla::host::launch_pdl(kernel, grid, block, 0, s, 0, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return MLA_OK;
}

}  // extern "C"

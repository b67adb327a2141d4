// Shared by the chunk attention and the attention mass: the layout of a CTA's
// score pipeline (page ring, queries in tensor memory, score buffers) and the
// move of a block's query rows from the ring into tensor memory.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "sm100_ptx.cuh"

namespace mla {
namespace chunk {

constexpr int kPage = 64;
constexpr int kDL = 512;
constexpr int kDR = 64;
constexpr int kRows = 128;    // rows per CTA
// warps: 0 TMA, 1 MMA, 2 TMEM alloc, 4-11 row warps (2, 3: query scales of an e4m3 cache, -lse of the mass)
constexpr int kThreads = 384;
constexpr int kMaxSB = 3;      // S buffers
constexpr int kCtrlBytes = 768;
constexpr int kMaxStages = 10;
constexpr int kMaxP = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMinusBig = -1.0e30f;  // running-maximum start (finite: no inf - inf)
// PV: f16 operands with an e4m3 cache, else bf16 (format 0 and 1 of kind::f16)
constexpr uint32_t make_idesc_pv(bool f16, uint32_t m) {
  return make_idesc(false, m, 256, false, true) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}

template <bool kF8, int kCg>
struct Cfg {
  // S CTA: a score tile is kCg pages, one 64-key page of it in each S CTA of
  // the pair (kCg = 2: one MMA covers N = 128 keys).  A page arrives in kParts
  // ring slots of kPartBoxes 128-byte columns each.
  static constexpr int kBox = 8192;                      // 64 rows x 128 bytes
  static constexpr int kSBoxes = kF8 ? 4 : 9;            // columns of a page in the 3-D box
  static constexpr int kPeBytes = kF8 ? 4096 : 0;        // e4m3 k_pe, 64-byte rows by a map of their own
  static constexpr int kParts = (kCg == 2 && !kF8) ? 3 : 1;
  static constexpr int kPartBoxes = kSBoxes / kParts;
  static constexpr int kSlotS = kPartBoxes * kBox + kPeBytes;
  static constexpr int kNStS = kF8 ? (kCg == 1 ? 6 : 5) : (kCg == 1 ? 3 : 7);
  static constexpr int kNTile = kParts == 3 ? 3 : kNStS;  // barriers that pages land on: tiles the ring can hold, or entries
  // TMEM columns: queries, then kNSB score buffers of a tile each.  A pair
  // keeps the rope part of the queries in shared memory (A of its QK steps),
  // which leaves 256 columns for two tiles of 128 keys.
  static constexpr bool kPeSmem = kCg == 2;
  static constexpr uint32_t kSCol0 = kCg == 1 ? 320 : 256;
  static constexpr int kNSB = kCg == 1 ? 3 : 2;
  static constexpr uint32_t kTileCols = 64 * kCg;
  static constexpr uint32_t kQLoCol = kCg == 1 ? 144 : 128;  // e4m3: the lo terms' first column
  // ring entries of a block's bf16 query rows.  bf16 pair: q_nope of 64 rows
  // like a page (parts of 3, 3 and 2 boxes; entry 2 part + half), q_pe
  // straight into its tile; else kQRows rows with q_pe as a ninth box
  static constexpr int kQRows = kParts == 3 ? 64 : kSlotS / 1152;
  static constexpr int kQEntries = kParts * kRows / kQRows;
  // O CTA: 512 / kCg latent dimensions of every page
  static constexpr int kVDims = kDL / kCg;
  static constexpr int kVBox = 8192;                     // 64 keys x 128 bytes
  static constexpr int kVBoxes = kVDims / 64;
  static constexpr int kSlotV = kVBoxes * kVBox;
  static constexpr int kNV = kF8 ? (kCg == 1 ? 2 : 3) : (kCg == 1 ? 3 : 4);
  static constexpr int kRawBoxes = kVDims / 128;         // e4m3: 64 keys x 128 codes
  static constexpr int kSlotRaw = kRawBoxes * kVBox;
  static constexpr int kNRaw = kF8 ? (kCg == 1 ? 2 : 3) : 0;
  static constexpr int kNStO = kF8 ? kNRaw : kNV;        // slots that TMA fills
  static constexpr int kSlotO = kF8 ? kSlotRaw : kSlotV;
  static constexpr int kNP = kCg == 1 ? 2 : 4;           // P slots
  static constexpr bool kVByP = !kF8 && kNP == kNV;      // a V slot is free when its page's P slot is
  static constexpr int kPBytes = kRows * kPage * 2;
  // P: K-major without swizzle, core matrices of 8 rows x 16 bytes; the
  // 16-byte chunk c of row r at (r / 8) * 1024 + c * 128 + (r % 8) * 16
  static constexpr uint32_t kPLbo = 128, kPSbo = 1024;
  static constexpr uint32_t kIdescQK = make_idesc(kF8, 128 * kCg, 64 * kCg, false, false);
  static constexpr uint32_t kIdescPV = make_idesc_pv(kF8, 128 * kCg);
  // shared memory
  // S: the rope parts of the queries (bf16: two units' tiles of 128 rows x
  // 128 bytes, swizzled by TMA; e4m3: hi and lo tiles of 128 rows x 64 codes)
  static constexpr int kQPeOff = kNStS * kSlotS;
  static constexpr int kQPeTile = kF8 ? 8192 : 16384;
  static constexpr int kMlOff = kQPeOff + (kPeSmem ? 2 * kQPeTile : 0);  // S: (m0, l0, m1, l1)[128]
  static constexpr int kPubOff = kMlOff + kRows * 16;    // S: row references of the last 4 pages
  static constexpr int kQsOff = kPubOff + 4 * kRows * 8;  // S, e4m3: two units' query scales
  static constexpr int kDataS = kQsOff + (kF8 ? 2 * kRows * 4 : 0);
  static constexpr int kVOff = kNP * kPBytes;            // O: P slots, V ring, raw ring, staging, row factors, flags
  static constexpr int kRawOff = kVOff + kNV * kSlotV;
  static constexpr int kStageOff = kRawOff + kNRaw * kSlotRaw;
  // per row warp of a pair's O CTA: its rows' sums as they come from the S
  // CTA, then boxes (2 KB) of outputs on their way to memory: two, or the one
  // that fits beside an e4m3 pair's rings
  static constexpr int kStage = kCg == 1 ? 0 : (kF8 ? 2048 : 4096);
  static constexpr int kRefOff = kStageOff + 8 * kStage;
  static constexpr int kFlagOff = kRefOff + kNP * kRows * 4;
  static constexpr int kDataO = kFlagOff + kNP * 16;
  static constexpr int kData = kDataS > kDataO ? kDataS : kDataO;
  static constexpr int kSmem = ((kData + 15) & ~15) + kCtrlBytes;  // at a 1024-byte boundary
  // bytes an S CTA sends per page: every row's P and O factor, a flag word per softmax warp
  static constexpr uint32_t kPTx = kRows * (kPage * 2 + 4) + 4 * 4;
  static constexpr uint32_t kMlTx = kRows * 16 * 2;  // per unit: every row's two (m, l), for the two warps of the row
  static constexpr int kCorrWarps = 8;  // O rows are corrected and stored by 8 warps, a half of the columns each
  static_assert(kSmem <= 232448, "shared memory budget");
  // Ring entries of a block with `rows` rows in the first CTA (the pair's CTAs
  // keep in step): as many as hold them.  Two units' entries are at least what
  // the ring holds, so that what unit n + 2 arms, unit n has released; a bf16
  // pair's rope tiles need one unit's entries to be that many.
  static constexpr int kMinQEntries = kParts == 3 ? kQEntries : (kNStS + 1) / 2 - kParts > 1 ? (kNStS + 1) / 2 - kParts : 1;
  static __device__ __forceinline__ int q_entries(int rows) {
    if (kParts == 3) return kQEntries;
    const int n = ((rows < kRows ? rows : kRows) + kQRows - 1) / kQRows;
    return n < kMinQEntries ? kMinQEntries : n;
  }
  static_assert(kQEntries <= kNStS && kNStS <= kMaxStages && 2 * (kMinQEntries + kParts) >= kNStS, "query entries");
  static_assert(kParts != 3 || kQEntries + kParts >= kNStS, "a pair's rope tiles");
};

// Where 16-byte chunk c of query row r of this CTA sits in the ring (c / 8:
// box, c % 8: piece of the 128-byte-swizzled row), first entry i.
template <bool kF8, int kCg>
__device__ __forceinline__ const uint8_t* q_chunk(const uint8_t* ring, uint32_t i, int r, int c) {
  using C = Cfg<kF8, kCg>;
  const int e = r / C::kQRows, rq = r % C::kQRows, box = c >> 3;
  const uint32_t entry = C::kParts == 3 ? i + 2 * (box / 3) + e : i + e;
  const int in_slot = C::kParts == 3 ? box % 3 : box;
  return ring + (entry % C::kNStS) * C::kSlotS + in_slot * (C::kQRows * 128) + rq * 128 + (((c & 7) ^ (rq & 7)) << 4);
}

// Query row r into TMEM lane r (bf16): 16-byte chunks [c0, c0 + kN).  The
// shared memory has been read when it returns; the stores need tmem_wait_st.
template <int kCg, int kN>
__device__ __forceinline__ void q_row_bf16(const uint8_t* ring, uint32_t i, int r, uint32_t taddr, int c0) {
  constexpr int kStep = kN % 12 == 0 ? 12 : 8;
#pragma unroll
  for (int c = 0; c < kN; c += kStep) {
    uint4 v[kStep];
#pragma unroll
    for (int k = 0; k < kStep; ++k) v[k] = *reinterpret_cast<const uint4*>(q_chunk<false, kCg>(ring, i, r, c0 + c + k));
#pragma unroll
    for (int s4 = 0; s4 < kStep / 4; ++s4) {
      const uint32_t w[16] = {v[4 * s4].x,     v[4 * s4].y,     v[4 * s4].z,     v[4 * s4].w,
                              v[4 * s4 + 1].x, v[4 * s4 + 1].y, v[4 * s4 + 1].z, v[4 * s4 + 1].w,
                              v[4 * s4 + 2].x, v[4 * s4 + 2].y, v[4 * s4 + 2].z, v[4 * s4 + 2].w,
                              v[4 * s4 + 3].x, v[4 * s4 + 3].y, v[4 * s4 + 3].z, v[4 * s4 + 3].w};
      tmem_st16(taddr + (c0 + c + 4 * s4) * 4, w);
    }
  }
}

// Two e4m3 codes, in the low bytes of the halves, as f16 values times 2^-8:
// moving exponent and mantissa to f16's place (exponent bias 15 instead of 7)
// scales every finite code by exactly 2^-8, subnormals included; the outputs'
// scale puts it back.  (b & 127) << 7 | (b & 128) << 8 = (b + (b & 128)) * 128,
// half of it on the multiply pipe; the conversion instruction took twice as
// long.  A NaN code becomes 1.875: its key's scores, from the codes as they
// are, are NaN already.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) { return b * 128u + (b & 0x00800080u) * 128u; }

// An e4m3 cache's scale of query row r: the power of two that puts the row's
// largest |q| into [2^7, 2^8) (2^-107 at least, so that its reciprocal stays
// finite); NaN for a row with an infinity or a NaN.
template <int kCg>
__device__ __forceinline__ float q_row_scale(const uint8_t* ring, uint32_t i, int r) {
  // the largest |q| (a NaN stays), two lanes in each of four chains
  __nv_bfloat162 m4[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) m4[e] = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll 6
  for (int c = 0; c < 72; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(q_chunk<true, kCg>(ring, i, r, c));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m4[e] = __hmax2_nan(m4[e], __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
  }
  const __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(m4[0], m4[1]), __hmax2_nan(m4[2], m4[3]));
  const uint32_t top = __bfloat16_as_ushort(__hmax_nan(m2.x, m2.y));
  int e = static_cast<int>(top >> 7) - 127 - 7;  // exponent of the scale
  e = e < -107 ? -107 : e;
  return __uint_as_float(top >= 0x7F80u ? 0x7FC00000u : static_cast<uint32_t>(e + 127) << 23);
}

// Query row r into TMEM for an e4m3 cache: the row as hi + lo e4m3 terms of
// q / scale; groups of 8 chunks [g0, g1), group 8 being the rope part, which a
// pair keeps in shared memory (K-major core matrices: the 16-byte chunk c of
// row r at (r / 8) * 512 + c * 128 + (r % 8) * 16).
template <int kCg>
__device__ __forceinline__ void q_row_e4m3(const uint8_t* ring, uint32_t i, int r, uint32_t taddr, uint8_t* pe_tile,
                                           int g0, int g1, float scale) {
  using C = Cfg<true, kCg>;
  // 1 / scale, a power of two in bf16 too (of a NaN an infinity: the row's scores are NaN by the scale)
  const uint32_t inv_bits = (254u - ((__float_as_uint(scale) >> 23) & 255u)) << 7 & 0x7F80u;
  const uint32_t inv_pair = inv_bits | (inv_bits << 16);
  const __nv_bfloat162 inv2 = *reinterpret_cast<const __nv_bfloat162*>(&inv_pair);
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(q_chunk<true, kCg>(ring, i, r, 8 * g + k));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          // q / scale is exact in bf16 and, from 2^-14 on, in f16 (8 bits, at
          // most 2^8); so is the residual of its e4m3 rounding
          const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * h2 + q]), inv2);
          const __half2 x = __float22half2_rn(__bfloat1622float2(y));
          const __nv_fp8x2_storage_t hh =
              __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&x), __NV_SATFINITE, __NV_E4M3);
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(hh, __NV_E4M3);
          const __half2 res = __hsub2(x, *reinterpret_cast<const __half2*>(&hr));
          h[q] = hh;
          l[q] = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&res), __NV_SATFINITE, __NV_E4M3);
        }
        hi[2 * k + h2] = h[0] | (h[1] << 16);
        lo[2 * k + h2] = l[0] | (l[1] << 16);
      }
    }
    if (C::kPeSmem && g == 8) {
      uint8_t* d = pe_tile + (r >> 3) * 512 + (r & 7) * 16;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        *reinterpret_cast<uint4*>(d + c * 128) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
        *reinterpret_cast<uint4*>(d + C::kQPeTile + c * 128) =
            make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
      }
    } else {
      tmem_st16(taddr + g * 16, hi);
      tmem_st16(taddr + C::kQLoCol + g * 16, lo);
    }
  }
  tmem_wait_st();
  if (C::kPeSmem) fence_proxy_async_cta();  // the rope tile is read by MMAs
}

}  // namespace chunk
}  // namespace mla

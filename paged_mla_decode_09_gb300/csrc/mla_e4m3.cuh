// Rounding to e4m3 codes of a value over a per-tensor scale, shared by the
// cache writes (mla_kv_pack.cu, mla_rope.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

namespace mla {
namespace e4m3 {

// Rounding x / scale to e4m3 without a division.  With r = fp32(1 /
// scale), x * r is within 2^-23 (relative) of x / scale; r_dn = fp32(r (1 -
// 2^-20)) and r_up = fp32(r (1 + 2^-20)) put x * r_dn and x * r_up on either
// side of x / scale.  When both round to the same code, so does the
// quotient (rounding is monotone); otherwise an e4m3 midpoint lies within
// about 2^-20 of it (rare) and e4m3_exact decides.
//
// e4m3_exact: the code nearest to x / scale.  m is the midpoint nearest q =
// x * r (the only one that x / scale can lie across), and x - m * scale,
// formed by one fma, has exactly the sign of x / scale - m for scale > 0
// (one rounding never changes a sign; only an exact zero is zero).  A value
// just past m on that side (or m itself on a tie, which the conversion
// sends to the even code) is then converted.  In e4m3's normal range (2^-6
// .. 448: 3 mantissa bits) the midpoints are the fp32 numbers whose
// mantissa bits 19..0 are 0x80000; the subnormal range [0, 2^-6) has the
// grid step of the binade [2^-6, 2^-5) (2^-9), so |q| + 2^-6 locates its
// midpoint there (g may round by at most 2^-30, which can move it across
// a code value but never across a midpoint, and the midpoint found on
// either side of a code value still separates x / scale from the code it
// does not round to).
static __device__ __noinline__ uint32_t e4m3_exact(float x, float scale, float inv_scale) {
  const float q = __fmul_rn(x, inv_scale);
  const float shift = fabsf(q) < 0x1p-6f ? 0x1p-6f : 0.f;
  const float g = fabsf(q) + shift;
  const float mi = __uint_as_float((__float_as_uint(g) & ~0xFFFFFu) | 0x80000u);
  const float m = copysignf(mi - shift, q);
  const float t = __fmaf_rn(-m, scale, x);
  const float v = t > 0.f ? m + fabsf(m) * 0x1p-10f : (t < 0.f ? m - fabsf(m) * 0x1p-10f : m);
  return static_cast<uint32_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}

struct Scale {
  float scale, r, r_dn, r_up;
};

// e4m3 codes of two bf16 values (packed as in memory, the lower address in
// the low half) times a factor: the lower address goes to the low byte
__device__ __forceinline__ uint32_t cvt2(uint32_t bf2, float f) {
  const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bf2));
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x.x, f), __fmul_rn(x.y, f)), __NV_SATFINITE, __NV_E4M3));
}

// the codes nearest to x / scale of the 8 bf16 values of a 16-byte chunk
__device__ __forceinline__ uint2 e4m3x8(uint4 v, const Scale& k) {
  const uint2 dn = make_uint2(cvt2(v.x, k.r_dn) | (cvt2(v.y, k.r_dn) << 16), cvt2(v.z, k.r_dn) | (cvt2(v.w, k.r_dn) << 16));
  const uint2 up = make_uint2(cvt2(v.x, k.r_up) | (cvt2(v.y, k.r_up) << 16), cvt2(v.z, k.r_up) | (cvt2(v.w, k.r_up) << 16));
  if (dn.x == up.x && dn.y == up.y) return dn;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
    c[e] = e4m3_exact(x.x, k.scale, k.r) | (e4m3_exact(x.y, k.scale, k.r) << 8);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// the codes nearest to x / scale of 8 fp32 values
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], const Scale& k) {
  uint32_t dn[4], up[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    dn[e] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(x[2 * e], k.r_dn), __fmul_rn(x[2 * e + 1], k.r_dn)), __NV_SATFINITE, __NV_E4M3));
    up[e] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(x[2 * e], k.r_up), __fmul_rn(x[2 * e + 1], k.r_up)), __NV_SATFINITE, __NV_E4M3));
    if (dn[e] != up[e]) dn[e] = e4m3_exact(x[2 * e], k.scale, k.r) | (e4m3_exact(x[2 * e + 1], k.scale, k.r) << 8);
  }
  return make_uint2(dn[0] | (dn[1] << 16), dn[2] | (dn[3] << 16));
}

// a normal, finite scale whose reciprocal is finite too
inline bool scale_ok(float kv_scale) {
  return kv_scale >= FLT_MIN && std::isfinite(kv_scale) && std::isfinite(1.0f / kv_scale);
}
inline Scale scale_of(float kv_scale) {
  Scale k;
  k.scale = kv_scale;
  k.r = 1.0f / kv_scale;  // IEEE fp32 division, once per call
  k.r_dn = k.r * (1.0f - 0x1p-20f);
  k.r_up = k.r * (1.0f + 0x1p-20f);
  return k;
}

}  // namespace e4m3
}  // namespace mla

// e4m3_quant.cuh — device helpers of the cache-writing kernels: group scales
// amax / 448 and the E4M3 codes of bf16 rows under them, both equal to the
// IEEE divisions bit for bit but without a division instruction (the kernels
// that use them are bound by instruction issue as much as by HBM).
#pragma once

#include <cstdint>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace smla {

// Two floats -> two E4M3 codes (RN, saturating): lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four E4M3 codes -> their values (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float& a, float& b, float& c, float& d) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(w));
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&lo));
  const float2 y = __half22float2(*reinterpret_cast<__half2*>(&hi));
  a = x.x; b = x.y; c = y.x; d = y.y;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// RN(amax / 448) without a division: amax * RN(1/448) is within an ulp and
// one fma residual correction (Markstein) rounds it; checked against the
// IEEE quotient for every positive finite bf16 amax (amax is a bf16 value).
__device__ __forceinline__ float amax_over_448(float amax) {
  constexpr float kInv = 1.f / 448.f;
  const float q0 = amax * kInv;
  if (!(amax <= 3.0e38f)) return q0;                 // inf: inf / 448
  return fmaf(fmaf(-q0, 448.f, amax), kInv, q0);
}

// RN(1/s) for a normal s: one Newton step from the hardware approximation
// (within an ulp); checked for the scale of every bf16 amax mantissa, from
// the approximation and from both of its fp32 neighbours.
__device__ __forceinline__ float recip_rn(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return fmaf(fmaf(-s, y, 1.f), y, y);
}

// Scales whose quotients the main path does not cover: below 2^-64 (the
// residual could lose bits to underflow), inf and NaN.  The largest finite
// scale (bf16 amax / 448) is below 2^120.
__device__ __forceinline__ bool special_scale(float s) {
  return !(s >= 0x1p-64f && s <= 0x1p120f);
}

// Quotients of 8 channels given as their negations xn (two per 64-bit word)
// with ny = -RN(1/s):
//   q0 = x * y,  u = q0 * s - x (exact, one fma),  q = q0 - u * y.
// q is RN(x / s) (Markstein: y the correctly rounded reciprocal, q0 within
// an ulp), checked for every bf16 x against every bf16 amax's scale.  The
// negated inputs make the signs of zeros come out as the division's.
__device__ __forceinline__ uint2 codes8(const uint64_t (&xn)[4], uint64_t s2, uint64_t ny2) {
  uint32_t c[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const uint64_t q0 = mul2(xn[p], ny2);
    const uint64_t u = fma2(q0, s2, xn[p]);
    float lo, hi;
    unpack2(fma2(u, ny2, q0), lo, hi);
    c[p] = e4m3x2(lo, hi);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// A 16-byte chunk of 8 bf16 -> their negations as 4 packed fp32 pairs, and
// the largest magnitude folded into amax.
__device__ __forceinline__ void unpack_neg8(const uint4 v, uint64_t (&xn)[4], float& amax) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float lo = __uint_as_float((w[p] << 16) ^ 0x80000000u);
    const float hi = __uint_as_float((w[p] & 0xFFFF0000u) ^ 0x80000000u);
    amax = fmaxf(amax, fmaxf(fabsf(lo), fabsf(hi)));
    xn[p] = pack2(lo, hi);
  }
}

// One chunk's codes for a special scale (the rare tail): a tiny scale and
// the chunk are first multiplied by 2^64 (the quotients are unchanged); inf
// and NaN scales give x * rcp(scale) (x / inf = +-0 for finite x, NaN for
// x = inf; x / NaN = NaN).
__device__ __forceinline__ uint2 special_codes8(const uint4 v, float s) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float q[8];
  if (s < 0x1p-64f) {
    const float ss = s * 0x1p64f;
    const float y = recip_rn(ss);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = e & 1 ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16);
      const float xn = -__uint_as_float(b) * 0x1p64f;
      const float q0 = xn * -y;
      q[e] = fmaf(fmaf(q0, ss, xn), -y, q0);
    }
  } else {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = e & 1 ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16);
      q[e] = __uint_as_float(b) * r;
    }
  }
  return make_uint2(e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16),
                    e4m3x2(q[4], q[5]) | (e4m3x2(q[6], q[7]) << 16));
}

}  // namespace smla

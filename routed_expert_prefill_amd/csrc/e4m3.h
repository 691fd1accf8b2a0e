// Encoding fp32 values as E4M3 codes under a row scale, shared by the row
// quantisation kernels and the norm that quantises its output.
#pragma once

#include "common.h"

namespace moe {

// fp32 -> E4M3FN code, round to nearest even, saturating |v| >= 448 to 448,
// sign of zero kept, NaN -> 0x7f.
__device__ __forceinline__ uint32_t f32_to_e4m3(float v) {
  const uint32_t b = __float_as_uint(v);
  const uint32_t sign = (b >> 24) & 0x80u;
  const uint32_t a = b & 0x7fffffffu;
  if (a > 0x7f800000u) return sign | 0x7fu;
  if (a >= 0x43e00000u) return sign | 0x7eu;  // 448.0f
  if (a >= 0x3c800000u) {                     // 2^-6: normal E4M3 range
    uint32_t r = a + 0x7ffffu + ((a >> 20) & 1u);  // RNE at the 4th significant bit
    r >>= 20;                                      // (exp32 << 3) | mantissa3
    return sign | (r - (120u << 3));               // rebias 127 -> 7
  }
  // subnormal range: multiples of 2^-9 (8 * 2^-9 = 2^-6 encodes as 0x08)
  const float s = __uint_as_float(a) * 512.0f;
  return sign | (uint32_t)__builtin_rintf(s);
}

// E4M3 codes of two fp32 values that are not NaN, in bytes 2 HI and 2 HI + 1
// of old: gfx950's conversion instruction (OCP E4M3FN, round to nearest
// even) on the values clamped to +-448.  On every fp32 pattern of magnitude
// below 464 it gives the same code as f32_to_e4m3 (subnormal codes and ties
// included; checked on MI355X), and from 464 on NaN, hence the clamp.
template <bool HI>
__device__ __forceinline__ uint32_t cvt_e4m3_x2(float a, float b, uint32_t old) {
  a = fminf(fmaxf(a, -448.0f), 448.0f);
  b = fminf(fmaxf(b, -448.0f), 448.0f);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
}

// q = e4m3_rne_saturate(fl32(v / sc)) without a division for nearly every
// element.  rcp = fl32(1 / sc); exact: the row needs the division throughout
// (sc not a normal float, or rcp not finite).
//
// y = v * rcp differs from fl32(v / sc) by a few units in the last place
// (two roundings of relative size 2^-24 each against one), i.e. by at most a
// handful of consecutive fp32 bit patterns.  E4M3 rounding is monotone and
// changes only at the midpoints between neighbouring codes, which in the
// normal range are the patterns whose low 20 bits are 0x80000.  So where y
// lies in the normal range and more than 16 patterns from a midpoint, the
// quotient has y's code.  Within that window (ties included), in the
// subnormal-code range, for NaN and for rows flagged exact the quotient is
// formed by IEEE division instead; the flag costs three compares, and the
// division runs behind one branch for the rare flagged elements.
__device__ __forceinline__ bool quant_needs_division(float y) {
  const uint32_t a = __float_as_uint(y) & 0x7fffffffu;
  return (a - 1u) < 0x3c7fffffu           // 0 < |y| < 2^-6: subnormal codes
         || a > 0x7f800000u               // NaN
         || ((a & 0xfffffu) - 0x7fff0u) < 32u;  // near a midpoint
}

// Four codes (one byte each) of v[0..3].  zero: the row is all zeros and
// every code is 0.
__device__ __forceinline__ uint32_t quant_e4m3_x4(const float (&v)[4], float sc, float rcp,
                                                  bool exact, bool zero) {
  float y[4];
  bool any = exact;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    y[e] = v[e] * rcp;
    any = any || quant_needs_division(y[e]);
  }
  uint32_t packed = cvt_e4m3_x2<false>(y[0], y[1], 0u);
  packed = cvt_e4m3_x2<true>(y[2], y[3], packed);
  if (any) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (exact || quant_needs_division(y[e]))
        packed = (packed & ~(0xffu << (8 * e))) | (f32_to_e4m3(v[e] / sc) << (8 * e));
    }
  }
  return zero ? 0u : packed;
}

// The same for the bf16 pairs lo and hi.
__device__ __forceinline__ uint32_t quant_e4m3_x4(uint32_t lo, uint32_t hi, float sc, float rcp,
                                                  bool exact, bool zero) {
  const float v[4] = {bf16_bits_to_f32((uint16_t)(lo & 0xffffu)),
                      bf16_bits_to_f32((uint16_t)(lo >> 16)),
                      bf16_bits_to_f32((uint16_t)(hi & 0xffffu)),
                      bf16_bits_to_f32((uint16_t)(hi >> 16))};
  return quant_e4m3_x4(v, sc, rcp, exact, zero);
}

// The scale of a row whose largest magnitude is amax.
__device__ __forceinline__ float q_scale(float amax) { return amax == 0.0f ? 1.0f : amax / 448.0f; }

// The reciprocal of a row scale, and whether the row must divide throughout.
__device__ __forceinline__ float quant_rcp(float sc, bool *exact) {
  const float r = 1.0f / sc;
  *exact = !(sc >= 1.17549435e-38f) || !(r < 3.40282347e38f);  // sc subnormal, r overflowed
  return r;
}

}  // namespace moe

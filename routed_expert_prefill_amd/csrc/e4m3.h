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

// ---- blocks of 128 columns, a scale for each ----

// amax / 448 of a block.  fp32 rows may be so small that the quotient rounds to
// zero: the smallest number then, so that codes stand for multiples of something.
__device__ __forceinline__ float qb_scale(float amax) {
  return amax == 0.0f ? 1.0f : fmaxf(amax / 448.0f, __uint_as_float(1u));
}

constexpr int kQbLanes = 16;  // lanes to a block, eight consecutive elements each

enum : int { kQbBf16 = 0, kQbF32 = 1 };

// Eight elements from element `at` of rows of the given kind.
template <int KIND>
__device__ __forceinline__ void qb_load(const void *x, size_t at, float (&v)[8]) {
  if constexpr (KIND == kQbBf16) {
    const i32x4 raw = *reinterpret_cast<const i32x4 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      v[2 * w] = __uint_as_float((uint32_t)raw[w] << 16);
      v[2 * w + 1] = __uint_as_float((uint32_t)raw[w] & 0xffff0000u);
    }
  } else {
    const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(x) + at);
    const f32x4 lo = p[0], hi = p[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = lo[e];
      v[4 + e] = hi[e];
    }
  }
}

// Correctly rounded quotients by fused multiply-adds, where `rcp` is 1 / d correctly
// rounded (qb_rcp): y = v rcp is within 1.5 steps of v / d, one step of refinement
// brings it within one, and a second rounds it correctly (Markstein's theorem; the
// residuals v - y d are exact).  d has no mantissa of ones only, and nothing here
// leaves the normal range: qb_plain.  The sign is v's: of v = -0 the sums are +0.
__device__ __forceinline__ float qb_div(float v, float d, float rcp) {
  float y = v * rcp;
  y = __builtin_fmaf(__builtin_fmaf(-y, d, v), rcp, y);
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-y, d, v), rcp, y), v);
}
// 1 / d of the same: the hardware's is within a step.
__device__ __forceinline__ float qb_rcp(float d) {
  const float y = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-y, d, 1.0f), y, y);
}
// Whether a block's scale, from its largest magnitude's bits, allows that.  The
// quotients of elements far below the largest may leave the normal range; their codes
// are zeros all the same, 2^-10 being the least that is none.
__device__ __forceinline__ bool qb_plain(uint32_t top, float sc) {
  return top - 0x20000000u < 0x40000000u  // 2^-63 .. 2^65
         && (__float_as_uint(sc) & 0x7fffffu) != 0x7fffffu;
}

template <int CTRL>
__device__ __forceinline__ uint32_t qb_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}

// Codes of the eight elements that a lane of a block's sixteen holds, and the
// block's scale, by the rule of quant.hip, except that a block of NaN, or of NaN and
// zeros, is not one of zeros: its scale is 1 as well, but a NaN keeps a NaN's code.
// All lanes of the wave call it together.
__device__ __forceinline__ uint2 qb_codes(const float (&v)[8], float *scale) {
  // the largest magnitude by its bits; a NaN's are above an infinity's
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = max(top, qb_dpp<0xb1>(top));   // lanes ^ 1
  top = max(top, qb_dpp<0x4e>(top));   // ^ 2
  top = max(top, qb_dpp<0x141>(top));  // 7 - lane, of eight
  top = max(top, qb_dpp<0x140>(top));  // 15 - lane, of sixteen
  float sc = qb_div(__uint_as_float(top), 448.0f, 1.0f / 448.0f);
  uint2 out = {0, 0};
  const bool plain = qb_plain(top, sc);
  if (plain) {
    const float rcp = qb_rcp(sc);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = qb_div(v[e], sc, rcp);
    out.x = cvt_e4m3_x2<true>(y[2], y[3], cvt_e4m3_x2<false>(y[0], y[1], 0u));
    out.y = cvt_e4m3_x2<true>(y[6], y[7], cvt_e4m3_x2<false>(y[4], y[5], 0u));
  }
  if (__any(!plain)) {  // zeros, NaN, infinities, very large and very small blocks
    float amax = 0.0f;  // which leaves NaN out
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
    for (int m = kQbLanes / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
    if (!plain) {
      const bool zero = top == 0;  // (amax is 0 of NaN too)
      sc = qb_scale(amax);
      bool exact;
      const float rcp = quant_rcp(sc, &exact);
      const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
      out.x = quant_e4m3_x4(lo, sc, rcp, exact, zero);
      out.y = quant_e4m3_x4(hi, sc, rcp, exact, zero);
    }
  }
  *scale = sc;
  return out;
}

}  // namespace moe

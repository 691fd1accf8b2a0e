// MXFP4 weights in registers: E2M1 codes, two to a byte (the earlier column
// in the low half), and one E8M0 scale (2^(byte - 127); 255 is NaN) for each
// 32 columns of a row.
//
// Every value below 2^128 that an E2M1 code and an E8M0 scale stand for is a
// bf16 number (subnormals included; larger ones become infinite), so gfx950's
// conversion instruction loses nothing and the products go through the bf16
// matrix unit: two weights per instruction, checked on MI355X for every byte
// under every scale.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// fp32 with the exponent field of an E8M0 scale: the conversion's operand.
__device__ __forceinline__ float mx4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight consecutive weights from the 32 bits that hold their codes.
__device__ __forceinline__ bf16x8 mx4_decode8(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

}  // namespace moe

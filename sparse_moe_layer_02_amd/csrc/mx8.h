// Blocks of 32 values in MXFP8 (e4m3 codes, one power-of-two scale byte a
// block), held by 4 neighbouring lanes of 8 values each.
#pragma once

#include "moe_internal.h"

namespace moe {
namespace mx8 {

typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
typedef __attribute__((__vector_size__(2 * sizeof(short)))) short s16x2;
typedef __attribute__((__vector_size__(2 * sizeof(unsigned)))) unsigned u32x2;

__device__ __forceinline__ float scale_of(unsigned byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);   // 0: 2^-127, a subnormal
}

// The codes of a lane's 8 values; byte: the scale of the block that they and
// the values of the lane's three neighbours make.  The largest magnitude is an
// integer maximum of the values' bits without sign, which ranks infinities and
// NaNs above every number.  With m = 2^e (1 + f) the scale is 2^(e - 8) up to
// 1 + f = 1.75 (m / scale <= 448), 2^(e - 7) above, so that nothing is clipped
// (a block's largest value of 1.75 to 2 times a power of two would lose up to
// an eighth of itself otherwise).
__device__ __forceinline__ u32x2 encode(const float* v, unsigned& byte) {
  unsigned top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
  top = max(top, (unsigned)__shfl_xor((int)top, 1));
  top = max(top, (unsigned)__shfl_xor((int)top, 2));
  // exponent field, one more where the mantissa passes 0.75
  const unsigned e = (top + 0x1fffffu) >> 23;
  byte = top >= 0x7f800000u ? 255u : e > 8 ? e - 8 : 0u;
  if (byte == 255u) return u32x2{0x7f7f7f7fu, 0x7f7f7f7fu};
  const float s = scale_of(byte);
  s16x2 a = {0, 0}, b = {0, 0};
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[0], v[1], s, false);
  a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[2], v[3], s, true);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[4], v[5], s, false);
  b = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(b, v[6], v[7], s, true);
  return u32x2{__builtin_bit_cast(unsigned, a), __builtin_bit_cast(unsigned, b)};
}

// The values of 8 codes of a block with this scale byte.
__device__ __forceinline__ void decode(u32x2 c, unsigned byte, float* v) {
  const float s = scale_of(byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[i], s, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[i], s, true);
    v[4 * i] = lo[0];
    v[4 * i + 1] = lo[1];
    v[4 * i + 2] = hi[0];
    v[4 * i + 3] = hi[1];
  }
}

}  // namespace mx8
}  // namespace moe

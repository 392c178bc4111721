// Blocks of 32 values in MXFP8 (e4m3 codes, one power-of-two scale byte a
// block), held by 4 neighbouring lanes of 8 values each or 8 lanes of 4.
#pragma once

#include <type_traits>

#include "wave.h"

namespace moe {
namespace mx8 {

typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
typedef __attribute__((__vector_size__(2 * sizeof(short)))) short s16x2;
typedef __attribute__((__vector_size__(2 * sizeof(unsigned)))) unsigned u32x2;

__device__ __forceinline__ float scale_of(unsigned byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);   // 0: 2^-127, a subnormal
}

// VEC codes, one to a byte.
template <int VEC> using Codes =
    std::conditional_t<VEC == 8, u32x2, std::conditional_t<VEC == 4, unsigned, void>>;

// The codes of a lane's VEC values; byte: the scale of the block that they and
// the values of the lane's neighbours, 32 / VEC lanes, make.  The largest magnitude is an
// integer maximum of the values' bits without sign, which ranks infinities and
// NaNs above every number.  With m = 2^e (1 + f) the scale is 2^(e - 8) up to
// 1 + f = 1.75 (m / scale <= 448), 2^(e - 7) above, so that nothing is clipped
// (a block's largest value of 1.75 to 2 times a power of two would lose up to
// an eighth of itself otherwise).
template <int VEC>
__device__ __forceinline__ Codes<VEC> encode(const float* v, unsigned& byte) {
  unsigned top = 0;
#pragma unroll
  for (int k = 0; k < VEC; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
  top = max(top, dpp_of<0xB1>(top));                   // lanes 1 apart
  top = max(top, dpp_of<0x4E>(top));                   // 2 apart
  if (VEC == 4) top = max(top, dpp_of<0x141>(top));    // the other four of eight
  // exponent field, one more where the mantissa passes 0.75
  const unsigned e = (top + 0x1fffffu) >> 23;
  byte = top >= 0x7f800000u ? 255u : e > 8 ? e - 8 : 0u;
  const float s = scale_of(byte == 255u ? 127u : byte);
  unsigned c[VEC / 4];
#pragma unroll
  for (int k = 0; k < VEC / 4; ++k) {
    s16x2 a = {0, 0};
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[4 * k], v[4 * k + 1], s, false);
    a = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(a, v[4 * k + 2], v[4 * k + 3], s, true);
    c[k] = byte == 255u ? 0x7f7f7f7fu : __builtin_bit_cast(unsigned, a);
  }
  if constexpr (VEC == 8)
    return u32x2{c[0], c[1]};
  else
    return c[0];
}

// The values of VEC codes of a block with this scale byte.
template <int VEC>
__device__ __forceinline__ void decode(Codes<VEC> codes, unsigned byte, float* v) {
  const float s = scale_of(byte);
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i) {
    unsigned c;
    if constexpr (VEC == 8)
      c = codes[i];
    else
      c = codes;
    const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, false);
    const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, s, true);
    v[4 * i] = lo[0];
    v[4 * i + 1] = lo[1];
    v[4 * i + 2] = hi[0];
    v[4 * i + 3] = hi[1];
  }
}

}  // namespace mx8
}  // namespace moe

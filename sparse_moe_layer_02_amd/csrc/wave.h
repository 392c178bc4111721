// Reductions over groups of W neighbouring lanes (8 to 64) on the data-parallel
// and lane-swap instructions: every lane of a group gets the same bits, and a
// step costs one or two instructions where a shuffle goes through LDS.
#pragma once

#include "moe_internal.h"

namespace moe {

template <int CTRL>
__device__ __forceinline__ float dpp_of(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}

template <int CTRL>
__device__ __forceinline__ unsigned dpp_of(unsigned v) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

// The values of the lanes 16 or 32 apart, as a pair whose order is the same for both.
__device__ __forceinline__ void swap16(float v, float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap32(float v, float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}

// op over a group: lanes 1 and 2 apart within fours, then fours and eights
// against each other mirrored (the lanes of each hold one value by then).
template <int W, typename Op>
__device__ __forceinline__ float group_reduce(float v, Op op) {
  v = op(v, dpp_of<0xB1>(v));                // quad_perm 1 0 3 2
  v = op(v, dpp_of<0x4E>(v));                // quad_perm 2 3 0 1
  v = op(v, dpp_of<0x141>(v));               // row_half_mirror
  if (W > 8) v = op(v, dpp_of<0x140>(v));    // row_mirror
  float a, b;
  if (W > 16) {
    swap16(v, a, b);
    v = op(a, b);
  }
  if (W > 32) {
    swap32(v, a, b);
    v = op(a, b);
  }
  return v;
}
template <int W>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<W>(v, [](float a, float b) { return a + b; });
}
template <int W>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<W>(v, [](float a, float b) { return fmaxf(a, b); });
}

}  // namespace moe

// Rows to MXFP4 and back (OCP Microscaling Formats (MX) v1.0: e2m1 codes, one
// e8m0 scale per 32 values).  Both are row sweeps bound by memory: rows are
// contiguous and a block of 32 never crosses one, so a sweep is over the flat
// array.  A lane takes 8 consecutive values (16 bytes of bf16, 32 of fp32) and
// 4 lanes a block; the largest magnitude is an integer maximum of the values'
// bits without sign, which ranks infinities and NaNs above every number and
// carries the exponent in place: scale byte = max(exponent field - 2, 0).
// Values are read and written past the caches (each is touched once): 65168 x
// 2048 bf16 values to codes and back to fp32, 0.94 GB, in 186 us before, 145
// with it; codes and scales keep the default policy, the product that follows
// reads them.
#include "block_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
typedef __attribute__((__vector_size__(2 * sizeof(float)))) float f32x2;
typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

__device__ __forceinline__ float scale_of(unsigned byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);   // 0: 2^-127, a subnormal
}

template <typename T> __device__ __forceinline__ void load8(const T* p, float* v);
template <> __device__ __forceinline__ void load8<bf16>(const bf16* p, float* v) {
  const bf16x8 x = __builtin_nontemporal_load((const bf16x8*)p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
}
template <> __device__ __forceinline__ void load8<float>(const float* p, float* v) {
  const f32x4 a = __builtin_nontemporal_load((const f32x4*)p);
  const f32x4 b = __builtin_nontemporal_load((const f32x4*)(p + 4));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// n8: groups of 8 values in all; n_rows bounds them by row8 groups a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void mxfp4_quantize(const T* __restrict__ x, long long n8,
                                                           const int32_t* __restrict__ n_rows,
                                                           int row8, uint32_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  long long end = n8;
  if (n_rows) end = min(end, (long long)max(*n_rows, 0) * row8);
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= end) return;   // rows hold whole blocks: all 4 lanes of a block or none
  float v[8];
  load8(x + i * 8, v);
  unsigned top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
  top = max(top, (unsigned)__shfl_xor((int)top, 1));
  top = max(top, (unsigned)__shfl_xor((int)top, 2));
  const unsigned e = top >> 23;
  const unsigned byte = e == 255 ? 255u : e > 2 ? e - 2 : 0u;
  const float s = scale_of(byte == 255 ? 127u : byte);
  unsigned c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  codes[i] = c;
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

// A lane stores 16 bytes at a time, a wave whole lines: bf16 lanes hold 8
// consecutive values, fp32 lanes 4, twice, 256 apart.  (8 consecutive fp32
// values a lane, half of every line in each store, lost what this gained.)
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_bf16(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long n8,
    bf16* __restrict__ y) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n8) return;
  const unsigned c = codes[i];
  const float s = scale_of(scales[i >> 2]);
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2);
  const bf16x2 f = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3);
  const bf16x8 v = {a[0], a[1], b[0], b[1], d[0], d[1], f[0], f[1]};
  __builtin_nontemporal_store(v, (bf16x8*)(y + i * 8));
}

__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_f32(
    const uint16_t* __restrict__ codes, const uint8_t* __restrict__ scales, long long n4,
    float* __restrict__ y) {
  const long long wave = (long long)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
  const long long first = wave * 2 * kWave + (threadIdx.x & (kWave - 1));
  unsigned c[2], e[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const long long i = first + u * kWave;
    if (i < n4) {
      c[u] = codes[i];
      e[u] = scales[i >> 3];
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const long long i = first + u * kWave;
    if (i < n4) {
      const float s = scale_of(e[u]);
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], s, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[u], s, 1);
      const f32x4 v = {a[0], a[1], b[0], b[1]};
      __builtin_nontemporal_store(v, (f32x4*)(y + i * 4));
    }
  }
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int dtype, long long rows, int cols,
                                 const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
  const long long n8 = rows * cols / 8;
  const unsigned grid = ceil_div((size_t)n8, kThreads);
  if (dtype == MOE_BF16)
    MOE_LAUNCH("mxfp4_quantize", s,
               mxfp4_quantize<bf16><<<grid, kThreads, 0, s>>>((const bf16*)x, n8, n_rows, cols / 8,
                                                              (uint32_t*)codes, scales));
  else
    MOE_LAUNCH("mxfp4_quantize", s,
               mxfp4_quantize<float><<<grid, kThreads, 0, s>>>((const float*)x, n8, n_rows,
                                                               cols / 8, (uint32_t*)codes,
                                                               scales));
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                   long long rows, int cols, void* y, hipStream_t s) {
  const long long n8 = rows * cols / 8;
  const unsigned grid = ceil_div((size_t)n8, kThreads);
  if (dtype == MOE_BF16)
    MOE_LAUNCH("mxfp4_dequantize", s,
               mxfp4_dequantize_bf16<<<grid, kThreads, 0, s>>>((const uint32_t*)codes, scales, n8,
                                                               (bf16*)y));
  else
    MOE_LAUNCH("mxfp4_dequantize", s,
               mxfp4_dequantize_f32<<<grid, kThreads, 0, s>>>((const uint16_t*)codes, scales,
                                                              2 * n8, (float*)y));
  return hipGetLastError();
}

}  // namespace moe

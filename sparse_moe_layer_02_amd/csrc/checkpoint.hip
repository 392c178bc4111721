// Activations in 8 bits between the forward and the backward pass: rows to
// MXFP8 and back, and the SwiGLU of the experts that writes its input in that
// form on the way and whose backward pass reads it there.
//   hh = g s u,  s = 1 / (1 + exp(-g));  d_u = d g s,  d_g = d u s (1 + g (1 - s))
// All are sweeps bound by memory.  A lane takes 8 consecutive values and 4
// lanes a block of 32; a block never crosses a row, and rows are contiguous.
#include "mx8.h"
#include "norm_rows.h"
#include "train_internal.h"

namespace moe {

using norms::Row8;

namespace {

constexpr int kThreads = 256;

// The first group behind the rows that count, of n groups, row8 a row.
__device__ __forceinline__ long long groups_end(long long n, const int32_t* n_rows, int row8) {
  return n_rows ? min(n, (long long)max(*n_rows, 0) * row8) : n;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mxfp8_quantize(const T* __restrict__ x, long long n8,
                                                           const int32_t* __restrict__ n_rows,
                                                           int row8, mx8::u32x2* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= groups_end(n8, n_rows, row8)) return;   // all 4 lanes of a block or none
  float v[8];
  Row8<T>::load(x + i * 8, v);
  unsigned byte;
  codes[i] = mx8::encode<8>(v, byte);
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mxfp8_dequantize(
    const mx8::u32x2* __restrict__ codes, const uint8_t* __restrict__ scales, long long n8,
    T* __restrict__ y) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n8) return;
  float v[8];
  mx8::decode<8>(codes[i], scales[i >> 2], v);
  Row8<T>::store(y + i * 8, v);
}

__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

// i: a group of 8 columns of the half, row8 a row.
template <typename T, bool SAVE>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(const T* __restrict__ gu, long long n8,
                                                          const int32_t* __restrict__ n_rows,
                                                          int row8, T* __restrict__ hh,
                                                          mx8::u32x2* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= groups_end(n8, n_rows, row8)) return;
  const long long at = i + i / row8 * row8;   // the gate's group; the up value's is row8 on
  float g[8], u[8], h[8];
  Row8<T>::load(gu + at * 8, g);
  Row8<T>::load(gu + (at + row8) * 8, u);
#pragma unroll
  for (int k = 0; k < 8; ++k) h[k] = g[k] * sigmoid(g[k]) * u[k];
  Row8<T>::store(hh + i * 8, h);
  if (SAVE) {
    unsigned byte;
    codes[at] = mx8::encode<8>(g, byte);
    if ((at & 3) == 0) scales[at >> 2] = (uint8_t)byte;
    codes[at + row8] = mx8::encode<8>(u, byte);
    if ((at & 3) == 0) scales[(at + row8) >> 2] = (uint8_t)byte;
  }
}

// d_gu may be gu and hh d_hh: a lane has read what it overwrites.
template <typename T, bool SAVED>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(
    const T* d_hh, const void* gu, const uint8_t* __restrict__ scales, long long n8,
    const int32_t* __restrict__ n_rows, int row8, T* d_gu, T* hh) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i >= groups_end(n8, n_rows, row8)) return;
  const long long at = i + i / row8 * row8;
  float d[8], g[8], u[8];
  Row8<T>::load(d_hh + i * 8, d);
  if (SAVED) {
    const mx8::u32x2* codes = (const mx8::u32x2*)gu;
    mx8::decode<8>(codes[at], scales[at >> 2], g);
    mx8::decode<8>(codes[at + row8], scales[(at + row8) >> 2], u);
  } else {
    Row8<T>::load((const T*)gu + at * 8, g);
    Row8<T>::load((const T*)gu + (at + row8) * 8, u);
  }
  float h[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float s = sigmoid(g[k]), a = g[k] * s;
    h[k] = a * u[k];
    const float dk = d[k];
    d[k] = dk * u[k] * (s + a * (1.0f - s));
    u[k] = dk * a;
  }
  Row8<T>::store(d_gu + at * 8, d);
  Row8<T>::store(d_gu + (at + row8) * 8, u);
  if (hh) Row8<T>::store(hh + i * 8, h);
}

}  // namespace

hipError_t launch_mxfp8_quantize(const void* x, int dtype, long long rows, int cols,
                                 const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
  const long long n8 = rows * cols / 8;
  const unsigned grid = ceil_div((size_t)n8, kThreads);
#define MX8_LAUNCH(T)                                                                       \
  MOE_LAUNCH("mxfp8_quantize", s,                                                           \
             mxfp8_quantize<T><<<grid, kThreads, 0, s>>>((const T*)x, n8, n_rows, cols / 8, \
                                                         (mx8::u32x2*)codes, scales))
  if (dtype == MOE_BF16)
    MX8_LAUNCH(bf16);
  else
    MX8_LAUNCH(float);
#undef MX8_LAUNCH
  return hipGetLastError();
}

hipError_t launch_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                   long long rows, int cols, void* y, hipStream_t s) {
  const long long n8 = rows * cols / 8;
  const unsigned grid = ceil_div((size_t)n8, kThreads);
#define MX8_LAUNCH(T)                                                                      \
  MOE_LAUNCH("mxfp8_dequantize", s,                                                        \
             mxfp8_dequantize<T><<<grid, kThreads, 0, s>>>((const mx8::u32x2*)codes, scales, \
                                                           n8, (T*)y))
  if (dtype == MOE_BF16)
    MX8_LAUNCH(bf16);
  else
    MX8_LAUNCH(float);
#undef MX8_LAUNCH
  return hipGetLastError();
}

hipError_t launch_swiglu(const void* gu, int dtype, long long rows, int I, const int32_t* n_rows,
                         void* hh, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const long long n8 = rows * (I / 8);
  const unsigned grid = ceil_div((size_t)n8, kThreads);
#define MX8_LAUNCH(T, SAVE)                                                                   \
  MOE_LAUNCH("swiglu", s,                                                                     \
             swiglu_kernel<T, SAVE><<<grid, kThreads, 0, s>>>((const T*)gu, n8, n_rows, I / 8, \
                                                              (T*)hh, (mx8::u32x2*)codes, scales))
  if (dtype == MOE_BF16) {
    if (codes)
      MX8_LAUNCH(bf16, true);
    else
      MX8_LAUNCH(bf16, false);
  } else {
    if (codes)
      MX8_LAUNCH(float, true);
    else
      MX8_LAUNCH(float, false);
  }
#undef MX8_LAUNCH
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const void* d_hh, const void* gu, const uint8_t* gu_scales,
                                  int dtype, long long rows, int I, const int32_t* n_rows,
                                  void* d_gu, void* hh, hipStream_t s) {
  const long long n8 = rows * (I / 8);
  const unsigned grid = ceil_div((size_t)n8, kThreads);
#define MX8_LAUNCH(T, SAVED)                                                                  \
  MOE_LAUNCH("swiglu_backward", s,                                                            \
             swiglu_backward_kernel<T, SAVED><<<grid, kThreads, 0, s>>>(                      \
                 (const T*)d_hh, gu, gu_scales, n8, n_rows, I / 8, (T*)d_gu, (T*)hh))
  if (dtype == MOE_BF16) {
    if (gu_scales)
      MX8_LAUNCH(bf16, true);
    else
      MX8_LAUNCH(bf16, false);
  } else {
    if (gu_scales)
      MX8_LAUNCH(float, true);
    else
      MX8_LAUNCH(float, false);
  }
#undef MX8_LAUNCH
  return hipGetLastError();
}

}  // namespace moe

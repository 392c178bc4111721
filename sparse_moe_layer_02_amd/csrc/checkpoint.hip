// Activations in 8 bits between the forward and the backward pass: rows to
// MXFP8 and back, and the SwiGLU of the experts that writes its input in that
// form on the way and whose backward pass reads it there.
//   hh = g s u,  s = 1 / (1 + exp(-g));  d_u = d g s,  d_g = d u s (1 + g (1 - s))
// All are sweeps bound by memory: a thread takes 8 values, as one piece or two,
// and the pieces of 32 / VEC neighbouring lanes are a block of 32 (a block never
// crosses a row, and rows are contiguous).  Everything goes past the caches but
// the codes that are written, which the backward pass finds there of a smaller
// batch, and the values that are converted alone, which another kernel has just
// written (8192 x 2048 fp32 13.0 us so, 15.7 past the caches; 8192 x 6144 bf16
// 28.4 and 27.3).  SwiGLU of 65387 rows of 2048 bf16 with its codes: 174 us each
// way, 6.2 TB/s (187 with the default policy).
#include "stream.h"
#include "train_internal.h"

namespace moe {

using namespace stream;

namespace {

constexpr int kThreads = 256;

// Groups of VEC values: group u of a thread.
template <int VEC> __device__ __forceinline__ long long group_of(int u) {
  return ((long long)blockIdx.x * (8 / VEC) + u) * kThreads + threadIdx.x;
}
// The first group behind the rows that count, of n groups, `row` a row.
__device__ __forceinline__ long long groups_end(long long n, const int32_t* n_rows, int row) {
  return n_rows ? min(n, (long long)max(*n_rows, 0) * row) : n;
}

// The codes of group g, and its block's scale byte.
template <int VEC>
__device__ __forceinline__ void store_codes(const float* v, long long g, uint8_t* codes,
                                            uint8_t* scales) {
  unsigned byte;
  ((mx8::Codes<VEC>*)codes)[g] = mx8::encode<VEC>(v, byte);
  if ((g & (32 / VEC - 1)) == 0) scales[g / (32 / VEC)] = (uint8_t)byte;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mxfp8_quantize(Source<T, piece_of<T>()> x,
                                                           long long n,
                                                           const int32_t* __restrict__ n_rows,
                                                           int row, uint8_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  constexpr int VEC = piece_of<T>();
  const long long end = groups_end(n, n_rows, row);
#pragma unroll
  for (int u = 0; u < 8 / VEC; ++u) {
    const long long g = group_of<VEC>(u);
    if (g < end) {   // all lanes of a block or none
      float v[VEC];
      Source<T, VEC>::values(*(const typename Source<T, VEC>::Raw*)(x.p + g * VEC), v);
      store_codes<VEC>(v, g, codes, scales);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void mxfp8_dequantize(Source<Mx8, piece_of<T>()> x,
                                                             long long n, T* __restrict__ y) {
  constexpr int VEC = piece_of<T>();
#pragma unroll
  for (int u = 0; u < 8 / VEC; ++u) {
    const long long g = group_of<VEC>(u);
    if (g < n) {
      float v[VEC];
      Source<Mx8, VEC>::values(x.load(g * VEC), v);
      store_past<VEC>(y + g * VEC, v);
    }
  }
}

// One form for both types, off by the few steps of exp, sum and quotient, which the
// sweeps hide behind memory: 0 from where exp(-g) passes 2^128, gates below -88.7.
__device__ __forceinline__ float sigmoid(float g) {
  return 1.0f / (1.0f + expf(-g));
}

// A group of VEC columns of the half, `row` a row.
template <typename T, bool SAVE>
__global__ __launch_bounds__(kThreads) void swiglu_kernel(Source<T, piece_of<T>()> gu,
                                                          unsigned n,
                                                          const int32_t* __restrict__ n_rows,
                                                          unsigned row, T* __restrict__ hh,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  constexpr int VEC = piece_of<T>();
  const long long end = groups_end(n, n_rows, row);
#pragma unroll
  for (int u = 0; u < 8 / VEC; ++u) {
    const long long i = group_of<VEC>(u);
    if (i < end) {
      // the gate's group; the up value's is `row` on
      const long long at = i + (long long)((unsigned)i / row) * row;
      const auto raw_g = gu.load(at * VEC), raw_u = gu.load((at + row) * VEC);
      float g[VEC], w[VEC], h[VEC];
      Source<T, VEC>::values(raw_g, g);
      Source<T, VEC>::values(raw_u, w);
#pragma unroll
      for (int k = 0; k < VEC; ++k) h[k] = g[k] * sigmoid(g[k]) * w[k];
      store_past<VEC>(hh + i * VEC, h);
      if (SAVE) {
        store_codes<VEC>(g, at, codes, scales);
        store_codes<VEC>(w, at + row, codes, scales);
      }
    }
  }
}

// X: T, or Mx8 of values kept in 8 bits.  d_gu may be gu and hh d_hh: a lane has
// read what it overwrites.
template <typename T, typename X>
__global__ __launch_bounds__(kThreads) void swiglu_backward_kernel(
    Source<T, piece_of<T>()> d_hh, Source<X, piece_of<T>()> gu, unsigned n,
    const int32_t* __restrict__ n_rows, unsigned row, T* d_gu, T* hh) {
  constexpr int VEC = piece_of<T>();
  const long long end = groups_end(n, n_rows, row);
#pragma unroll
  for (int u = 0; u < 8 / VEC; ++u) {
    const long long i = group_of<VEC>(u);
    if (i < end) {
      const long long at = i + (long long)((unsigned)i / row) * row;
      const auto raw_d = d_hh.load(i * VEC);
      const auto raw_g = gu.load(at * VEC), raw_u = gu.load((at + row) * VEC);
      float d[VEC], g[VEC], w[VEC], h[VEC];
      Source<T, VEC>::values(raw_d, d);
      Source<X, VEC>::values(raw_g, g);
      Source<X, VEC>::values(raw_u, w);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const float s = sigmoid(g[k]), a = g[k] * s, dk = d[k];
        h[k] = a * w[k];
        d[k] = dk * w[k] * (s + a * (1.0f - s));
        w[k] = dk * a;
      }
      store_past<VEC>(d_gu + at * VEC, d);
      store_past<VEC>(d_gu + (at + row) * VEC, w);
      if (hh) store_past<VEC>(hh + i * VEC, h);
    }
  }
}

}  // namespace

// Blocks of kThreads threads that have 8 values each.
static unsigned blocks_of(long long values) { return ceil_div((size_t)values / 8, kThreads); }

hipError_t launch_mxfp8_quantize(const void* x, int dtype, long long rows, int cols,
                                 const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s) {
#define MX8_LAUNCH(T)                                                                          \
  MOE_LAUNCH("mxfp8_quantize", s,                                                              \
             mxfp8_quantize<T><<<blocks_of(rows * cols), kThreads, 0, s>>>(                    \
                 {(const T*)x}, rows * cols / piece_of<T>(), n_rows, cols / piece_of<T>(), codes, \
                 scales))
  if (dtype == MOE_BF16)
    MX8_LAUNCH(bf16);
  else
    MX8_LAUNCH(float);
#undef MX8_LAUNCH
  return hipGetLastError();
}

hipError_t launch_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                   long long rows, int cols, void* y, hipStream_t s) {
#define MX8_LAUNCH(T)                                                          \
  MOE_LAUNCH("mxfp8_dequantize", s,                                            \
             mxfp8_dequantize<T><<<blocks_of(rows * cols), kThreads, 0, s>>>(  \
                 {codes, scales}, rows * cols / piece_of<T>(), (T*)y))
  if (dtype == MOE_BF16)
    MX8_LAUNCH(bf16);
  else
    MX8_LAUNCH(float);
#undef MX8_LAUNCH
  return hipGetLastError();
}

hipError_t launch_swiglu(const void* gu, int dtype, long long rows, int I, const int32_t* n_rows,
                         void* hh, uint8_t* codes, uint8_t* scales, hipStream_t s) {
#define MX8_LAUNCH(T, SAVE)                                                                 \
  MOE_LAUNCH("swiglu", s,                                                                   \
             swiglu_kernel<T, SAVE><<<blocks_of(rows * I), kThreads, 0, s>>>(               \
                 {(const T*)gu}, (unsigned)(rows * I / piece_of<T>()), n_rows,              \
                 I / piece_of<T>(), (T*)hh, codes, scales))
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
#define MX8_LAUNCH(T, X, ...)                                                                 \
  MOE_LAUNCH("swiglu_backward", s,                                                            \
             swiglu_backward_kernel<T, X><<<blocks_of(rows * I), kThreads, 0, s>>>(           \
                 {(const T*)d_hh}, __VA_ARGS__, (unsigned)(rows * I / piece_of<T>()), n_rows, \
                 I / piece_of<T>(), (T*)d_gu, (T*)hh))
  if (dtype == MOE_BF16) {
    if (gu_scales)
      MX8_LAUNCH(bf16, Mx8, {(const uint8_t*)gu, gu_scales});
    else
      MX8_LAUNCH(bf16, bf16, {(const bf16*)gu});
  } else {
    if (gu_scales)
      MX8_LAUNCH(float, Mx8, {(const uint8_t*)gu, gu_scales});
    else
      MX8_LAUNCH(float, float, {(const float*)gu});
  }
#undef MX8_LAUNCH
  return hipGetLastError();
}

}  // namespace moe

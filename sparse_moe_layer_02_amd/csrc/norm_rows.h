// What the row sweeps of the norms share: 8-element pieces of a row in fp32,
// sums over the threads of a row, the root of its mean square, and the shape of
// a launch over rows.
#pragma once

#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace norms {

constexpr int kMaxThreads = 1024;
constexpr unsigned kMaxGridX = 1u << 21;   // blocks of at most kMaxThreads

template <typename T> struct Row8;
template <> struct Row8<bf16> {
  static __device__ __forceinline__ void load(const bf16* p, float* o) {
    const bf16x8 v = *(const bf16x8*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = (float)v[i];
  }
  static __device__ __forceinline__ void store(bf16* p, const float* o) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (bf16)o[i];
    *(bf16x8*)p = v;
  }
};
template <> struct Row8<float> {
  static __device__ __forceinline__ void load(const float* p, float* o) {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = a[i];
      o[4 + i] = b[i];
    }
  }
  static __device__ __forceinline__ void store(float* p, const float* o) {
    *(f32x4*)p = f32x4{o[0], o[1], o[2], o[3]};
    *(f32x4*)(p + 4) = f32x4{o[4], o[5], o[6], o[7]};
  }
};

// Sum of v over the threads of a row; every one of them gets it.  part: 16
// floats of LDS of this sum alone.
__device__ __forceinline__ float row_sum(float v, float* part, bool one_wave) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  if (one_wave) return v;
  const int wave = threadIdx.x / kWave, n = blockDim.x / kWave;
  if ((threadIdx.x & (kWave - 1)) == 0) part[wave] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < n; ++w) v += part[w];
  return v;
}

// 1 / sqrt(mean(v^2) + eps) of a row whose threads hold the sums ss of their
// v's squares.  Squares past 2^128 leave no sum, and below 2^-126 they lose
// digits (which counts where eps does not cover them): such a row's v, rare and
// the same for all its threads, are scaled by a power of two, eps by its
// square, and summed again.  The scaled v times the root is the norm as before.
// part: two sums' LDS.
template <int P>
__device__ __forceinline__ float inv_rms(float (&v)[P][8], float ss, float eps, int H,
                                         float (*part)[kMaxThreads / kWave], bool one_wave) {
  float sum = row_sum(ss, part[0], one_wave);
  const bool large = !(sum < __builtin_inff()), small = sum < 0x1p-90f && eps < 0x1p-100f;
  if (large || small) {
    const float f = large ? 0x1p-96f : 0x1p96f;
    ss = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if ((p * (int)blockDim.x + (int)threadIdx.x) * 8 < H) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[p][i] *= f;
          ss = fmaf(v[p][i], v[p][i], ss);
        }
      }
    }
    sum = row_sum(ss, part[1], one_wave);
    eps = eps * f * f;
  }
  return rsqrtf(sum / (float)H + eps);
}

// The row of a thread.  The grid is a rectangle of blocks in row order.
__device__ __forceinline__ unsigned row_of_thread() {
  return (blockIdx.y * gridDim.x + blockIdx.x) * blockDim.y + threadIdx.y;
}

struct Shape {
  int P;
  dim3 block, grid;
};
// Rows of up to 2048 values take one piece a thread, up to 16384 two, up to
// 32768 four.  (8192 rows of 6144, residual in fp32: 113.5 us, 5.3 TB/s, with
// two pieces; with one 3 % more.)
inline Shape shape(int T, int H) {
  Shape s;
  s.P = H <= 2048 ? 1 : H <= 16 * kMaxThreads ? 2 : 4;
  const int per = ((H + 8 * s.P - 1) / (8 * s.P) + kWave - 1) / kWave * kWave;
  const int rows = per == kWave ? 4 : 1;
  s.block = dim3(per, rows);
  // a launch takes fewer than 2^32 threads along a dimension of its grid
  const unsigned blocks = ceil_div(T, rows);
  s.grid.x = std::min(blocks, kMaxGridX);
  s.grid.y = ceil_div(blocks, s.grid.x);
  return s;
}

}  // namespace norms
}  // namespace moe

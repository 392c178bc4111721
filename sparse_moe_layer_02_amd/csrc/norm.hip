// The norms before and after a block (root mean square), the second fused with
// the block's gate and residual scale, the residual sum and the next block's
// norm.
//   z = y * rsqrt(mean(y^2) + eps) * w_post;  s = residual + scale * gate * z
//   next = s * rsqrt(mean(s^2) + eps) * w_next
// Row sweeps bound by memory: each row is read once into registers (8-element
// pieces, P of them a thread), its sum of squares is taken in fp32 (a fixed
// order: bitwise the same from run to run), and the second norm works on the
// sums still in registers, so a row costs its inputs and outputs and no more.
// A row of at most 512 values is one wave's and needs no barrier, four such
// rows to a block; longer ones are a block's.
#include "block_internal.h"
#include "norm_rows.h"

namespace moe {

using namespace norms;

namespace {

// blockDim (threads of a row, rows of a block); one_wave: 64 threads a row.
template <typename T, typename U, int P>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(const T* x, const float* __restrict__ w,
                                                           float eps, int rows, int H, U* y) {
  __shared__ float part[2][kMaxThreads / kWave];
  const bool one_wave = blockDim.x == kWave;
  const unsigned t = row_of_thread();
  if (t >= (unsigned)rows) return;   // a whole wave, and then blocks have no barrier
  float v[P][8];
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      Row8<T>::load(x + (size_t)t * H + h, v[p]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[p][i], v[p][i], ss);
    }
  }
  const float r = inv_rms(v, ss, eps, H, part, one_wave);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      float g[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (w) Row8<float>::load(w + h, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = v[p][i] * r * g[i];
      Row8<U>::store(y + (size_t)t * H + h, v[p]);
    }
  }
}

template <typename Y, typename S, int P>
__global__ __launch_bounds__(kMaxThreads) void norm_residual_kernel(
    const Y* y, const float* __restrict__ w_post, float eps, const float* __restrict__ gate,
    int gate_kind, float scale, const S* residual, S* res_out, const float* __restrict__ w_next,
    Y* next, int rows, int H) {
  __shared__ float part[4][kMaxThreads / kWave];
  const bool one_wave = blockDim.x == kWave;
  const unsigned t = row_of_thread();
  if (t >= (unsigned)rows) return;
  float v[P][8], s[P][8];
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      Row8<Y>::load(y + (size_t)t * H + h, v[p]);
      Row8<S>::load(residual + (size_t)t * H + h, s[p]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[p][i], v[p][i], ss);
    }
  }
  float r = scale;
  if (gate_kind == MOE_GATE_TOKEN) r *= gate[t];
  if (w_post) r *= inv_rms(v, ss, eps, H, part, one_wave);
  ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      float g[8];
      if (w_post) {
        Row8<float>::load(w_post + h, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] *= g[i];
      }
      if (gate_kind == MOE_GATE_CHANNEL) {
        Row8<float>::load(gate + h, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] *= g[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[p][i] = fmaf(v[p][i], r, s[p][i]);
        ss = fmaf(s[p][i], s[p][i], ss);
      }
      Row8<S>::store(res_out + (size_t)t * H + h, s[p]);
    }
  }
  if (!next) return;
  r = inv_rms(s, ss, eps, H, part + 2, one_wave);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      float g[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (w_next) Row8<float>::load(w_next + h, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[p][i] = s[p][i] * r * g[i];
      Row8<Y>::store(next + (size_t)t * H + h, s[p]);
    }
  }
}

template <typename T, typename U>
void norm_t(const void* x, const float* w, float eps, int T_, int H, void* y, hipStream_t st) {
  const Shape s = shape(T_, H);
#define MX_NORM(P)                                                                            \
  MOE_LAUNCH("norm", st,                                                                      \
             norm_kernel<T, U, P><<<s.grid, s.block, 0, st>>>((const T*)x, w, eps, T_, H, (U*)y))
  if (s.P == 1)
    MX_NORM(1);
  else if (s.P == 2)
    MX_NORM(2);
  else
    MX_NORM(4);
#undef MX_NORM
}

template <typename Y, typename S>
void residual_t(const void* y, const float* w_post, float eps, const float* gate, int gate_kind,
                float scale, const void* residual, void* res_out, const float* w_next, void* next,
                int T, int H, hipStream_t st) {
  const Shape s = shape(T, H);
#define MX_NORM(P)                                                                            \
  MOE_LAUNCH("norm_residual", st,                                                             \
             norm_residual_kernel<Y, S, P><<<s.grid, s.block, 0, st>>>(                       \
                 (const Y*)y, w_post, eps, gate, gate_kind, scale, (const S*)residual,        \
                 (S*)res_out, w_next, (Y*)next, T, H))
  if (s.P == 1)
    MX_NORM(1);
  else if (s.P == 2)
    MX_NORM(2);
  else
    MX_NORM(4);
#undef MX_NORM
}

}  // namespace

hipError_t launch_norm(const void* x, int x_dtype, const float* weight, float eps, int T, int H,
                       void* y, int y_dtype, hipStream_t s) {
  if (x_dtype == MOE_BF16)
    y_dtype == MOE_BF16 ? norm_t<bf16, bf16>(x, weight, eps, T, H, y, s)
                        : norm_t<bf16, float>(x, weight, eps, T, H, y, s);
  else
    y_dtype == MOE_BF16 ? norm_t<float, bf16>(x, weight, eps, T, H, y, s)
                        : norm_t<float, float>(x, weight, eps, T, H, y, s);
  return hipGetLastError();
}

hipError_t launch_norm_residual(const void* y, int y_dtype, const float* w_post, float eps,
                                const float* gate, int gate_kind, float scale,
                                const void* residual, int res_dtype, void* res_out,
                                const float* w_next, void* next, int T, int H, hipStream_t s) {
#define MX_RES(Y, S)                                                                            \
  residual_t<Y, S>(y, w_post, eps, gate, gate_kind, scale, residual, res_out, w_next, next, T,  \
                   H, s)
  if (y_dtype == MOE_BF16)
    res_dtype == MOE_BF16 ? MX_RES(bf16, bf16) : MX_RES(bf16, float);
  else
    res_dtype == MOE_BF16 ? MX_RES(float, bf16) : MX_RES(float, float);
#undef MX_RES
  return hipGetLastError();
}

}  // namespace moe

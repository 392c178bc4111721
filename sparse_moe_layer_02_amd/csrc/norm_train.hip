// The norm by mean and variance, the norms that keep their input in 8 bits, and
// the backward pass of both norms.  With n = d r, d = x - m (the root mean
// square norm: m = 0), r = 1 / sqrt(mean(d^2) + eps) and g = dy weight:
//   y  = n weight + bias
//   dx = r (g - mean(g) - n mean(g n)) + d_residual    (root mean square: no mean(g))
//   d_weight = sum over rows of dy n,  d_bias = sum over rows of dy
// Row sweeps bound by memory, as in norm.hip: a row is read once into registers
// and the sums over it are taken there; the backward pass takes the row's
// statistics again instead of reading them, from the x that it needs anyway.
// Its blocks go over many rows each and keep the weights' gradients of their
// rows in registers, or in LDS on long rows; the blocks' sums are joined by a
// second kernel in a fixed order.
#include <type_traits>

#include "norm_rows.h"
#include "stream.h"
#include "train_internal.h"

namespace moe {

using namespace norms;
using namespace stream;

namespace {

constexpr int kMaxWaves = kMaxThreads / kWave;

// Sums of N values over the threads of a row.  part: LDS of their own, zero
// where there are fewer than WAVES waves.
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*part)[WAVES]) {
  const int waves = blockDim.x / kWave, lane = threadIdx.x & (kWave - 1);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = group_sum<kWave>(v[k]);
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[k][threadIdx.x / kWave] = v[k];
  }
  lds_barrier();   // loads of the next row stay in flight
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (WAVES == 4) {
      const f32x4 a = *(const f32x4*)part[k];
      v[k] = (a[0] + a[1]) + (a[2] + a[3]);
    } else {
      v[k] = group_sum<16>(part[k][lane & 15]);
    }
  }
}

// Rows whose sums leave fp32's range, as inv_rms has them.
__device__ __forceinline__ bool too_large(float ss) { return !(ss < __builtin_inff()); }
__device__ __forceinline__ bool too_small(float ss, float eps) {
  return ss < 0x1p-90f && eps < 0x1p-100f;
}

// Pieces of a row in a thread: piece p starts at at[p].  Only the last pieces,
// kLoose of them, may lie behind the row (row_shape sees to it): in[] for those.
// Loads are made for all pieces, from the row's start for one that is behind: a
// load under a condition would be waited for where it is made, to be merged
// with what was there.
template <int P, int VEC> struct Pieces {
  static constexpr int kLoose = 8 / VEC, kFirst = P - kLoose;
  int at[P];
  bool in[kLoose];
  __device__ __forceinline__ Pieces(int H) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      at[p] = (p * (int)blockDim.x + (int)threadIdx.x) * VEC;
      if (p >= kFirst) {
        in[p - kFirst] = at[p] < H;
        if (at[p] >= H) at[p] = 0;
      }
    }
  }
  __device__ __forceinline__ bool inside(int p) const { return p < kFirst || in[p - kFirst]; }
  // behind the row: nothing to any sum
  __device__ __forceinline__ void clear_behind(float (&v)[P][VEC]) const {
#pragma unroll
    for (int p = kFirst; p < P; ++p)
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[p][i] = in[p - kFirst] ? v[p][i] : 0.0f;
  }
};

// 8 values of a row in the order in which norm_kernel has them.
template <typename T> struct Eight;
template <> struct Eight<bf16> : Source<bf16, 8> {
  __device__ __forceinline__ Raw load(size_t at) const { return *(const Raw*)(p + at); }
};
template <> struct Eight<float> {
  struct Raw {
    f32x4 a, b;
  };
  const float* p;
  static __device__ __forceinline__ void arrived(Raw& r) {
    asm volatile("" : "+v"(r.a), "+v"(r.b));
  }
  // (through the caches: each load has half of its lines)
  __device__ __forceinline__ Raw load(size_t at) const {
    return Raw{*(const f32x4*)(p + at), *(const f32x4*)(p + at + 4)};
  }
  static __device__ __forceinline__ void values(const Raw& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = r.a[i];
      v[4 + i] = r.b[i];
    }
  }
};

// The root mean square norm that keeps its input: y is that of norm_kernel, bit
// for bit (the same threads hold the same values and join their sums in the
// same order), and a row's pieces of 4 neighbouring threads are a block of 32.
// A block goes over several rows with the weight in registers and, up to 16384
// values, the next row in flight: taken from L2 for every row, the weight's 4
// bytes a value were as much as x, y and the codes together (8192 x 6144 bf16:
// 47 us so, 42 now).
template <typename T, typename U, int P>
__global__ __launch_bounds__(kMaxThreads) void norm_checkpoint_kernel(
    Eight<T> x, const float* __restrict__ w, float eps, int rows, int H, U* y,
    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr bool kAhead = P <= 2;
  __shared__ float part[4][kMaxWaves];
  const bool one_wave = blockDim.x == kWave;
  const long long step = (long long)gridDim.x * blockDim.y;
  long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const Pieces<P, 8> pieces(H);
  typename Eight<T>::Raw next[P];
  const auto fetch = [&](long long row) {
    const size_t start = (size_t)min(row, (long long)rows - 1) * H;
#pragma unroll
    for (int p = 0; p < P; ++p) next[p] = x.load(start + pieces.at[p]);
  };
  if (kAhead) fetch(t);
  float g[P][8];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[p][i] = 1.0f;
    if (w) Row8<float>::load(w + pieces.at[p], g[p]);
  }
  const auto arrived = [&]() {
#pragma unroll
    for (int p = 0; p < P; ++p) Eight<T>::arrived(next[p]);
  };
  if (kAhead) arrived();
  int turn = 0;   // the sums of one row are read while those of the next are written
  for (; t < rows; t += step, turn ^= 2) {
    const size_t row = (size_t)t * H;
    float v[P][8];
    float ss = 0.0f;
    if (!kAhead) fetch(t);
#pragma unroll
    for (int p = 0; p < P; ++p) Eight<T>::values(next[p], v[p]);
    if (kAhead) fetch(t + step);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      unsigned byte;
      const mx8::Codes<8> c = mx8::encode<8>(v[p], byte);
      if (pieces.inside(p)) {
        const size_t at = row + pieces.at[p];
        *(mx8::Codes<8>*)(codes + at) = c;
        if ((threadIdx.x & 3) == 0) scales[at / 32] = (uint8_t)byte;
      }
    }
    pieces.clear_behind(v);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[p][i], v[p][i], ss);
    const float r = inv_rms(v, ss, eps, H, part + turn, one_wave);
    // the next row's loads end here, so that nothing waits for this row's stores
    if (kAhead) arrived();
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = v[p][i] * r * g[p][i];
      // past the caches, which then have the codes for the backward pass (113 -> 110 us
      // both ways, 8192 x 6144); fp32 in pieces of 8 would be half lines
      if (pieces.inside(p)) {
        if constexpr (std::is_same<U, bf16>::value)
          store_past<8>(y + row + pieces.at[p], v[p]);
        else
          Row8<U>::store(y + row + pieces.at[p], v[p]);
      }
    }
  }
}

// v = v - mean(v), but for the roundings of the mean's sum, which are not small
// beside the deviations where a row is far from zero (nor none where its values are
// equal: 3 v is no fp32 number for most v).
// over: divides a sum by the row's length, or multiplies it by the reciprocal, which
// is a rounding more and saves a backward pass of 16384 x 2048 bf16 4 %.
struct Length {
  float h;
  __device__ __forceinline__ float operator()(float sum) const { return sum / h; }
};
struct Reciprocal {
  float inv;
  __device__ __forceinline__ float operator()(float sum) const { return sum * inv; }
};
template <int WAVES, int P, int VEC, typename Over>
__device__ __forceinline__ void center(float (&v)[P][VEC], const Pieces<P, VEC>& pieces,
                                       Over over, float (*part)[WAVES]) {
  float s[1] = {0.0f};
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[0] += v[p][i];
  row_sums<WAVES>(s, part);
  const float m = over(s[0]);
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[p][i] -= m;
  pieces.clear_behind(v);
}

// The sum of v's squares.
template <int WAVES, int P, int VEC>
__device__ __forceinline__ float squares(const float (&v)[P][VEC], float (*part)[WAVES]) {
  float s[1] = {0.0f};
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s[0] = fmaf(v[p][i], v[p][i], s[0]);
  row_sums<WAVES>(s, part);
  return s[0];
}

template <int P, int VEC> __device__ __forceinline__ void scale(float (&v)[P][VEC], float f) {
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[p][i] *= f;
}

// What center() has left of the mean is alike for the whole row and of the
// deviations' own size.  Their mean m, summed with their squares, is taken out of
// the deviations where they are multiplied, and out of the squares' sum here.
// (Without it rows of 6144 values of mean 1000 and spread 1 were off by 1e-4, and
// equal values of 1000, which are normed to zeros, by up to 0.2.)  mostly: it is so
// much of the squares that what stays of them may be roundings alone.
struct Mean {
  float m, ss;
  bool mostly;
};
__device__ __forceinline__ Mean mean_left(float sum, float ss, float inv_h) {
  const float m = sum * inv_h, of_mean = sum * m;
  return {m, ss - of_mean, of_mean >= 0.0625f * ss && m != 0.0f};   // (both may be underflowed)
}

// Of the sum of squares as it was summed.
__device__ __forceinline__ float scale_of_row(float ss, float eps) {
  return too_large(ss) ? 0x1p-96f : too_small(ss, eps) ? 0x1p96f : 1.0f;
}

// The deviations of a row's values v, and the sum of their squares, where this left
// fp32's range or the mean had most of it: rare, and the same for the row's
// threads.  f: the power of two that they are scaled by, before the first mean is
// taken where it is less than 1, behind it otherwise.  Three means, as the second has a
// rounding of the first's error, which counts where the row is all but constant;
// deviations of equal values have few digits, so that their sum is exact and they
// become zeros, whose root is eps's alone: f's square would lose it.
// part: 4 sums' LDS.
template <int WAVES, int P, int VEC>
__device__ __forceinline__ float deviations(float (&v)[P][VEC], const Pieces<P, VEC>& pieces,
                                            int H, float& f, float (*part)[WAVES]) {
  const bool large = f < 1.0f;
  if (large) scale(v, f);
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {
    center(v, pieces, Length{(float)H}, part + k);
    if (k == 0 && !large) scale(v, f);
  }
  const float ss = squares(v, part + 3);
  if (large && ss == 0.0f) f = 1.0f;
  return ss;
}

// SAVE: x in 8 bits to codes and scales too; the pieces of 32 / VEC neighbouring
// threads are a block.  A block goes over the rows blockIdx.x * blockDim.y +
// threadIdx.y, and so on; up to 12288 values its threads have weight and bias in
// registers and the next row in flight.  (From L2 for every row, the two were
// more than x and y together: 8192 x 6144 fp32 to bf16 55.7 us so, 48.6 now.)
template <typename T, typename U, int P, int VEC, int THREADS, bool SAVE>
__global__ __launch_bounds__(THREADS) void layer_norm_kernel(
    Source<T, VEC> x, const float* __restrict__ w, const float* __restrict__ b, float eps,
    int rows, int H, U* y, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr bool kAhead = THREADS <= 512;
  constexpr int kWaves = THREADS <= 256 ? 4 : 16;
  constexpr int kSums = 7;
  __shared__ __attribute__((aligned(16))) float part[kSums][kWaves];
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < kSums * kWaves;
       i += blockDim.x * blockDim.y)
    (&part[0][0])[i] = 0.0f;
  __syncthreads();
  const long long step = (long long)gridDim.x * blockDim.y;
  long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const Pieces<P, VEC> pieces(H);
  const float inv_h = 1.0f / (float)H;
  typedef typename Source<T, VEC>::Raw Raw;
  Raw next[P];
  // (the last row where there is no next one)
  const auto fetch = [&](long long row) {
    const size_t start = (size_t)min(row, (long long)rows - 1) * H;
#pragma unroll
    for (int p = 0; p < P; ++p) next[p] = x.load(start + pieces.at[p]);
  };
  if (kAhead) fetch(t);
  float weight[kAhead ? P : 1][VEC], bias[kAhead ? P : 1][VEC];
  const auto affine = [&](int p, float* g, float* c) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      g[i] = 1.0f;
      c[i] = 0.0f;
    }
    if (w) load_floats<VEC>(w + pieces.at[p], g);
    if (b) load_floats<VEC>(b + pieces.at[p], c);
  };
  if (kAhead) {
#pragma unroll
    for (int p = 0; p < P; ++p) affine(p, weight[p], bias[p]);
#pragma unroll
    for (int p = 0; p < P; ++p) Source<T, VEC>::arrived(next[p]);
  }
  for (; t < rows; t += step) {
    const size_t row = (size_t)t * H;
    float v[P][VEC];
    if (!kAhead) fetch(t);
#pragma unroll
    for (int p = 0; p < P; ++p) Source<T, VEC>::values(next[p], v[p]);
    if (kAhead) fetch(t + step);
    if (SAVE) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        unsigned byte;
        const mx8::Codes<VEC> c = mx8::encode<VEC>(v[p], byte);
        if (pieces.inside(p)) {   // all lanes of a block or none
          const size_t at = row + pieces.at[p];
          *(mx8::Codes<VEC>*)(codes + at) = c;
          if (pieces.at[p] % 32 == 0) scales[at / 32] = (uint8_t)byte;
        }
      }
    }
    pieces.clear_behind(v);
    center(v, pieces, Reciprocal{inv_h}, part);
    float s[2] = {0.0f, 0.0f};   // the deviations' squares, and themselves
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        s[0] = fmaf(v[p][i], v[p][i], s[0]);
        s[1] += v[p][i];
      }
    row_sums<kWaves>(s, part + 1);
    Mean left = mean_left(s[1], s[0], inv_h);
    float f = scale_of_row(s[0], eps);
    if (left.mostly || f != 1.0f) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const Raw again = x.load(row + pieces.at[p]);
        Source<T, VEC>::values(again, v[p]);
      }
      pieces.clear_behind(v);
      left.ss = deviations(v, pieces, H, f, part + 3);
      left.m = 0.0f;
    }
    const float r = rsqrtf(left.ss * inv_h + eps * f * f), mr = left.m * r;
    // the next row's loads end here, so that nothing waits for this row's stores
    if (kAhead) {
#pragma unroll
      for (int p = 0; p < P; ++p) Source<T, VEC>::arrived(next[p]);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float g[VEC], c[VEC];
      if (!kAhead) affine(p, g, c);
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        v[p][i] = fmaf(fmaf(v[p][i], r, -mr), kAhead ? weight[p][i] : g[i],
                       kAhead ? bias[p][i] : c[i]);
      if (pieces.inside(p)) store_past<VEC>(y + row + pieces.at[p], v[p]);
    }
  }
}

// A block goes over the rows blockIdx.x * blockDim.y + threadIdx.y, and so on.
// sum_w, sum_b: the block's sums over its rows go to row blockIdx.x of them,
// `stride` floats a row; NULL: not asked for.
// Up to 12288 values a row's threads have the weight in registers and the next
// row's x and dy in flight while one is worked on: what a row costs once (its
// sums, addresses) is shared by up to 24 values a lane, and the blocks of a CU
// wait for different things.  (8192 x 6144, bf16 gradients, fp32 stream: 115 us,
// 6.1 TB/s; bf16 from 8-bit rows 62 us, 5.7.)  Longer rows have neither, and their 32
// values a lane do not fit 128 registers (2048 x 16384: 268 us, 1.8 TB/s).
template <typename DY, typename X, typename DX, int P, int VEC, int THREADS, bool MEAN>
__global__ __launch_bounds__(THREADS, THREADS <= 512 ? 2 : 1) void norm_backward_kernel(
    Source<DY, VEC> dy, Source<X, VEC> x, const float* __restrict__ w, float eps, int rows, int H,
    Source<DX, VEC> d_residual, DX* dx, float* __restrict__ sum_w, float* __restrict__ sum_b,
    int stride) {
  constexpr bool kAhead = THREADS <= 512;
  constexpr int kSums = MEAN ? 13 : 5, kWaves = THREADS <= 256 ? 4 : 16;
  // the weights' gradients of a thread's columns: in registers, or, where these
  // do not hold them for two waves a SIMD, in LDS that is the thread's alone
  constexpr bool kInLds = kAhead && P * VEC > 16;
  __shared__ __attribute__((aligned(16))) float acc[kInLds ? 2 : 1][kInLds ? P : 1]
                                                   [kInLds ? THREADS : 1][VEC];
  // the sums of one row are read while those of the next are written
  __shared__ __attribute__((aligned(16))) float part[2][kSums][kWaves];
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 2 * kSums * kWaves;
       i += blockDim.x * blockDim.y)
    (&part[0][0][0])[i] = 0.0f;
  __syncthreads();
  const long long step = (long long)gridDim.x * blockDim.y;
  long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const Pieces<P, VEC> pieces(H);
  const float inv_h = 1.0f / (float)H;
  float dw[P][VEC] = {}, db[P][VEC] = {};
  if (kInLds) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      store_floats<VEC>(acc[0][p][threadIdx.x], dw[p]);
      store_floats<VEC>(acc[1][p][threadIdx.x], db[p]);
    }
  }
  float weight[kAhead ? P : 1][VEC];
  const auto weights = [&](int p, float (&g)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = 1.0f;
    if (w) load_floats<VEC>(w + pieces.at[p], g);
  };
  typename Source<DY, VEC>::Raw next_dy[P];
  typename Source<X, VEC>::Raw next_x[P];
  // (from the last row where there is no next one)
  const auto fetch = [&](long long row) {
    const size_t start = (size_t)min(row, (long long)rows - 1) * H;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      next_x[p] = x.load(start + pieces.at[p]);
      next_dy[p] = dy.load(start + pieces.at[p]);
    }
  };
  const auto arrived = [&]() {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      Source<X, VEC>::arrived(next_x[p]);
      Source<DY, VEC>::arrived(next_dy[p]);
    }
  };
  if (kAhead) {
#pragma unroll
    for (int p = 0; p < P; ++p) weights(p, weight[p]);
    fetch(t);
    arrived();
  }
  for (int turn = 0; t < rows; t += step, turn ^= 1) {
    const size_t row = (size_t)t * H;
    float v[P][VEC], d[P][VEC];   // x, then its deviations; dy
    typename Source<DX, VEC>::Raw res[P];
    if (!kAhead) fetch(t);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      Source<X, VEC>::values(next_x[p], v[p]);
      Source<DY, VEC>::values(next_dy[p], d[p]);
    }
    if (d_residual.p) {
#pragma unroll
      for (int p = 0; p < P; ++p) res[p] = d_residual.load(row + pieces.at[p]);
    }
    if (kAhead) fetch(t + step);
    pieces.clear_behind(v);
    pieces.clear_behind(d);
    float s[4];
    // the squares of v, g times v, g, and v
    const auto sums = [&](float (*lds)[kWaves]) {
      s[0] = s[1] = s[2] = s[3] = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float g[VEC];
        if (!kAhead) weights(p, g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float gi = d[p][i] * (kAhead ? weight[p][i] : g[i]);
          s[0] = fmaf(v[p][i], v[p][i], s[0]);
          s[1] = fmaf(gi, v[p][i], s[1]);
          if (MEAN) {
            s[2] += gi;
            s[3] += v[p][i];
          }
        }
      }
      if (MEAN) {
        row_sums<kWaves>(s, lds);
      } else {
        float two[2] = {s[0], s[1]};
        row_sums<kWaves>(two, lds);
        s[0] = two[0];
        s[1] = two[1];
      }
    };
    float (*lds)[kWaves] = part[turn];
    const auto own = [&](int n) {   // LDS of the next n sums
      float (*at)[kWaves] = lds;
      lds += n;
      return at;
    };
    if (MEAN) center(v, pieces, Reciprocal{inv_h}, own(1));
    sums(own(MEAN ? 4 : 2));
    Mean left = {0.0f, s[0], false};
    if (MEAN) {
      left = mean_left(s[3], s[0], inv_h);
      s[1] = fmaf(-left.m, s[2], s[1]);
    }
    // n = (v - m) to_n, dx = (..) root half
    float f = scale_of_row(s[0], eps), root = rsqrtf(left.ss * inv_h + eps), to_n = root;
    float half = 1.0f;
    if (left.mostly || f != 1.0f || !(fabsf(s[1]) < __builtin_inff())) {
      // rare, and the same for the row's threads: v scaled, then normed before it meets g
#pragma unroll
      for (int p = 0; p < P; ++p) Source<X, VEC>::values(x.load(row + pieces.at[p]), v[p]);
      pieces.clear_behind(v);
      float ss;
      if (MEAN) {
        ss = deviations(v, pieces, H, f, own(4));
        left.m = 0.0f;
      } else {
        scale(v, f);
        ss = squares(v, own(1));
      }
      root = rsqrtf(ss * inv_h + eps * f * f);
      scale(v, root);
      to_n = 1.0f;
      sums(own(MEAN ? 4 : 2));
      // f in two halves: neither root f nor (..) root is sure to be one of fp32's numbers
      half = f < 1.0f ? 0x1p-48f : f > 1.0f ? 0x1p48f : 1.0f;
      root *= half;
    }
    // the next row's loads end here, so that nothing waits for this row's stores
    if (kAhead) arrived();
    const float c = to_n * s[1] * inv_h, mean_g = MEAN ? s[2] * inv_h : 0.0f,
                mn = left.m * to_n;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float g[VEC], o[VEC] = {};
      if (!kAhead) weights(p, g);
      if (d_residual.p) Source<DX, VEC>::values(res[p], o);
      if (kInLds) {
        load_floats<VEC>(acc[0][p][threadIdx.x], dw[p]);
        load_floats<VEC>(acc[1][p][threadIdx.x], db[p]);
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float n = MEAN ? fmaf(v[p][i], to_n, -mn) : v[p][i] * to_n;
        const float gi = d[p][i] * (kAhead ? weight[p][i] : g[i]);
        o[i] = fmaf((gi - mean_g - n * c) * root, half, o[i]);
        dw[p][i] = fmaf(d[p][i], n, dw[p][i]);
        db[p][i] += d[p][i];
      }
      if (kInLds) {
        store_floats<VEC>(acc[0][p][threadIdx.x], dw[p]);
        if (MEAN) store_floats<VEC>(acc[1][p][threadIdx.x], db[p]);
      }
      if (pieces.inside(p)) store_past<VEC>(dx + row + pieces.at[p], o);
    }
  }
  if (!sum_w && !sum_b) return;
  if (P * VEC == 8 && blockDim.y > 1) {
    // the block's rows at a time share a column: joined in their order
    __shared__ float other[3][2][kWave * 8];
    if (threadIdx.y > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          other[threadIdx.y - 1][0][(p * VEC + i) * kWave + threadIdx.x] = dw[p][i];
          other[threadIdx.y - 1][1][(p * VEC + i) * kWave + threadIdx.x] = db[p][i];
        }
    }
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dw[p][i] += other[y - 1][0][(p * VEC + i) * kWave + threadIdx.x];
          db[p][i] += other[y - 1][1][(p * VEC + i) * kWave + threadIdx.x];
        }
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (pieces.inside(p)) {
      if (kInLds) {
        load_floats<VEC>(acc[0][p][threadIdx.x], dw[p]);
        load_floats<VEC>(acc[1][p][threadIdx.x], db[p]);
      }
      const size_t to = (size_t)blockIdx.x * stride + pieces.at[p];
      if (sum_w) store_floats<VEC>(sum_w + to, dw[p]);
      if (MEAN && sum_b) store_floats<VEC>(sum_b + to, db[p]);
    }
}

// Eight loads in flight a thread (256 rows of 6144, weight and bias: 5 us; one at a
// time 12).  d[h] = sum over n rows of sums[.][h], 64 columns a block; blockIdx.y: the
// weight's sums, then the bias's, H floats behind them.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(kWave* kJoinWaves) void join_sums(const float* __restrict__ sums,
                                                               int n, int stride, int H,
                                                               float* __restrict__ d_weight,
                                                               float* __restrict__ d_bias) {
  __shared__ float part[kJoinWaves][kWave];
  float* out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int wave = threadIdx.y, h = blockIdx.x * kWave + threadIdx.x;
  float v = 0.0f;
  if (h < H) {
    const float* p = sums + blockIdx.y * H + h;
    for (int k0 = wave; k0 < n; k0 += 8 * kJoinWaves) {
      float a[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int k = k0 + u * kJoinWaves;
        a[u] = k < n ? p[(size_t)k * stride] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) v += a[u];
    }
  }
  part[wave][threadIdx.x] = v;
  __syncthreads();
  if (wave > 0 || h >= H) return;
  for (int k = 1; k < kJoinWaves; ++k) v += part[k][threadIdx.x];
  out[h] = v;
}

// Blocks that go over rows, per_cu of them a CU but for no more than 32 waves.
void bound_blocks(Shape& s, int T, unsigned per_cu) {
  const unsigned most = 32 * kWave / (s.block.x * s.block.y);
  s.grid = dim3(std::min(ceil_div(T, s.block.y), 256 * std::max(1u, std::min(per_cu, most))));
}
// Threads of a row, P pieces of 8 values each: up to 6144 values at most 256
// threads, four rows of a wave to a block where that is enough for one; up to
// 12288 at most 512.  (P - 1) * 8 values for every thread lie inside the row:
// Pieces counts on it.
Shape row_shape(int H) {
  Shape s;
  s.P = H <= 6144 ? ceil_div(H, 2048) : H <= 12288 ? ceil_div(H, 4096) : 4;
  const int per = ceil_div(ceil_div(H, 8 * s.P), kWave) * kWave;
  s.block = dim3(per, per == kWave ? 4 : 1);
  return s;
}
// The forward pass: as many blocks as have up to 32 KB of rows at a time (with
// the next ones in flight as much again).  More of them read and write in more
// places at once and are slower, fewer leave the memory idle: 8192 x 6144 fp32
// 49 us with one block of 24 KB, 51 with four; 16384 x 2048 51 with one of 8 KB, 34
// with four.
Shape forward_shape(int T, int H, int x_bytes) {
  Shape s = row_shape(H);
  bound_blocks(s, T, 32768 / (H * x_bytes * s.block.y));
  return s;
}
// The backward pass: as few blocks as have 20 KB of loads at a time, for the same
// reason (8192 x 6144 with fp32 rows 121 us with one block, 129 with two; 16384 x
// 2048 bf16 68 with one of 12 KB, 53 with two, 55 with three), and each block's
// sums are written and read again.  bytes: of a value in all that is read.
Shape backward_shape(int T, int H, int bytes) {
  Shape s = row_shape(H);
  bound_blocks(s, T, ceil_div(20480, H * bytes * s.block.y));
  return s;
}
constexpr int kLeastBytes = 4;   // dy and x of 16 bits, no residual

}  // namespace

size_t norm_backward_ws_bytes(int T, int H) {
  return (size_t)backward_shape(T, H, kLeastBytes).grid.x * 2 * H * sizeof(float);
}

namespace {

// CALL(P, THREADS) for a row shape.
#define MOE_ROW_P(H, s, CALL)   \
  if ((H) <= 6144) {            \
    if ((s).P == 1)             \
      CALL(1, 256);             \
    else if ((s).P == 2)        \
      CALL(2, 256);             \
    else                        \
      CALL(3, 256);             \
  } else if ((H) <= 12288) {    \
    if ((s).P == 2)             \
      CALL(2, 512);             \
    else                        \
      CALL(3, 512);             \
  } else {                      \
    CALL(4, 1024);              \
  }

template <typename T, typename U>
void checkpoint_t(const void* x, const float* w, float eps, int T_, int H, void* y,
                  uint8_t* codes, uint8_t* scales, hipStream_t st) {
  Shape s = shape(T_, H);
  bound_blocks(s, T_, std::max(2u, 32768u / (H * (unsigned)sizeof(T) * s.block.y)));
#define MOE_NORM(P)                                                                       \
  MOE_LAUNCH("norm_checkpoint", st,                                                       \
             norm_checkpoint_kernel<T, U, P><<<s.grid, s.block, 0, st>>>(                 \
                 Eight<T>{(const T*)x}, w, eps, T_, H, (U*)y, codes, scales))
  if (s.P == 1)
    MOE_NORM(1);
  else if (s.P == 2)
    MOE_NORM(2);
  else
    MOE_NORM(4);
#undef MOE_NORM
}

template <typename T, typename U>
void layer_norm_t(const void* x, const float* w, const float* b, float eps, int T_, int H,
                  void* y, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const Shape s = forward_shape(T_, H, sizeof(T));
  constexpr int VEC = piece_of<T, U>();
#define MOE_NORM(P, THREADS, SAVE)                                                            \
  MOE_LAUNCH("layer_norm", st,                                                                \
             layer_norm_kernel<T, U, P * 8 / VEC, VEC, THREADS, SAVE>                         \
                 <<<s.grid, s.block, 0, st>>>(Source<T, VEC>{(const T*)x}, w, b, eps, T_, H, \
                                              (U*)y, codes, scales))
#define MOE_SAVE(P, THREADS) MOE_NORM(P, THREADS, true)
#define MOE_PLAIN(P, THREADS) MOE_NORM(P, THREADS, false)
  if (codes) {
    MOE_ROW_P(H, s, MOE_SAVE)
  } else {
    MOE_ROW_P(H, s, MOE_PLAIN)
  }
#undef MOE_PLAIN
#undef MOE_SAVE
#undef MOE_NORM
}

// x: the rows or codes, x_scales with codes.
template <typename X, int VEC> Source<X, VEC> source_of(const void* x, const uint8_t* x_scales) {
  if constexpr (std::is_same<X, Mx8>::value)
    return Source<X, VEC>{(const uint8_t*)x, x_scales};
  else
    return Source<X, VEC>{(const X*)x};
}

template <typename DY, typename X, typename DX>
void backward_t(bool mean, const void* dy, const void* x, const uint8_t* x_scales, const float* w,
                float eps, int T, int H, const void* d_residual, void* dx, float* d_weight,
                float* d_bias, float* ws, hipStream_t st) {
  // (8-bit rows count as the bf16 ones that hold the same: their sums are the same bits)
  constexpr int kX = std::is_same<X, float>::value ? 4 : 2;
  Shape s = backward_shape(T, H, (int)sizeof(DY) + kX + (d_residual ? (int)sizeof(DX) : 0));
  // A few rows are one block's, which has the whole sums: 8.2 us a call for 4 to 16
  // rows of 256 and 1 to 4 of 2048 values, with a launch that joins the sums of
  // more blocks 10.7 to 11.0.  On the GPU alone the fifth row in turn (of 6144
  // values the third) takes longer than that launch.
  if ((d_weight || d_bias) && s.grid.x <= (H <= 4096 ? 4 : 2)) s.grid.x = 1;
  constexpr int VEC = piece_of<DY, X, DX>();
  // one block has the whole sums
  const bool join = s.grid.x > 1 && (d_weight || d_bias);
  float* sum_w = join ? ws : d_weight;
  float* sum_b = join ? ws + H : d_bias;
#define MOE_NORM(P, THREADS, MEAN)                                                            \
  MOE_LAUNCH("norm_backward", st,                                                             \
             norm_backward_kernel<DY, X, DX, P * 8 / VEC, VEC, THREADS, MEAN>                 \
                 <<<s.grid, s.block, 0, st>>>(                                                \
                     Source<DY, VEC>{(const DY*)dy}, source_of<X, VEC>(x, x_scales), w, eps, T, \
                     H, Source<DX, VEC>{(const DX*)d_residual}, (DX*)dx, sum_w, sum_b, 2 * H))
#define MOE_MEAN(P, THREADS) MOE_NORM(P, THREADS, true)
#define MOE_ROOT(P, THREADS) MOE_NORM(P, THREADS, false)
  if (mean) {
    MOE_ROW_P(H, s, MOE_MEAN)
  } else {
    MOE_ROW_P(H, s, MOE_ROOT)
  }
#undef MOE_ROOT
#undef MOE_MEAN
#undef MOE_NORM
  if (join)
    MOE_LAUNCH("norm_join_sums", st,
               join_sums<<<dim3(ceil_div(H, kWave), mean ? 2 : 1), dim3(kWave, kJoinWaves), 0,
                           st>>>(ws, s.grid.x, 2 * H, H, d_weight, d_bias));
}

template <typename DY, typename DX>
void backward_x(bool mean, const void* dy, const void* x, int x_dtype, const uint8_t* x_scales,
                const float* w, float eps, int T, int H, const void* d_residual, void* dx,
                float* d_weight, float* d_bias, float* ws, hipStream_t st) {
#define MOE_BACK(X)                                                                         \
  backward_t<DY, X, DX>(mean, dy, x, x_scales, w, eps, T, H, d_residual, dx, d_weight, d_bias, \
                        ws, st)
  if (x_scales)
    MOE_BACK(Mx8);
  else if (x_dtype == MOE_BF16)
    MOE_BACK(bf16);
  else
    MOE_BACK(float);
#undef MOE_BACK
}

}  // namespace

hipError_t launch_norm_save(bool mean, const void* x, int x_dtype, const float* weight,
                            const float* bias, float eps, int T, int H, void* y, int y_dtype,
                            uint8_t* codes, uint8_t* scales, hipStream_t s) {
#define MOE_SAVE(T_, U)                                                                \
  (mean ? layer_norm_t<T_, U>(x, weight, bias, eps, T, H, y, codes, scales, s)         \
        : checkpoint_t<T_, U>(x, weight, eps, T, H, y, codes, scales, s))
  if (x_dtype == MOE_BF16)
    y_dtype == MOE_BF16 ? MOE_SAVE(bf16, bf16) : MOE_SAVE(bf16, float);
  else
    y_dtype == MOE_BF16 ? MOE_SAVE(float, bf16) : MOE_SAVE(float, float);
#undef MOE_SAVE
  return hipGetLastError();
}

hipError_t launch_norm_backward(bool mean, const void* dy, int dy_dtype, const void* x,
                                int x_dtype, const uint8_t* x_scales, const float* weight,
                                float eps, int T, int H, const void* d_residual, void* dx,
                                int dx_dtype, float* d_weight, float* d_bias, void* ws,
                                hipStream_t s) {
#define MOE_BACK(DY, DX)                                                                       \
  backward_x<DY, DX>(mean, dy, x, x_dtype, x_scales, weight, eps, T, H, d_residual, dx, d_weight, \
                     d_bias, (float*)ws, s)
  if (dy_dtype == MOE_BF16)
    dx_dtype == MOE_BF16 ? MOE_BACK(bf16, bf16) : MOE_BACK(bf16, float);
  else
    dx_dtype == MOE_BF16 ? MOE_BACK(float, bf16) : MOE_BACK(float, float);
#undef MOE_BACK
  return hipGetLastError();
}

}  // namespace moe

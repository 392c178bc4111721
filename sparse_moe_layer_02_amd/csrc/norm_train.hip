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
// rows in registers; the blocks' sums are joined by a second kernel in a fixed
// order.
#include "mx8.h"
#include "norm_rows.h"
#include "train_internal.h"
#include "wave.h"

namespace moe {

using namespace norms;

namespace {

constexpr int kMaxWaves = kMaxThreads / kWave;

// A row's 8 values as they are kept: loaded early as Raw, taken apart later.
// arrived: a point that the load is waited for at, before any that follow it.
template <typename T> struct Source;
template <> struct Source<bf16> {
  typedef bf16x8 Raw;
  const bf16* p;
  static __device__ __forceinline__ void arrived(Raw& r) { asm volatile("" : "+v"(r)); }
  __device__ __forceinline__ Raw load(size_t at) const { return *(const bf16x8*)(p + at); }
  static __device__ __forceinline__ void values(const Raw& r, float* v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)r[i];
  }
};
template <> struct Source<float> {
  struct Raw {
    f32x4 a, b;
  };
  const float* p;
  static __device__ __forceinline__ void arrived(Raw& r) {
    asm volatile("" : "+v"(r.a), "+v"(r.b));
  }
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
struct Mx8;
template <> struct Source<Mx8> {
  struct Raw {
    mx8::u32x2 codes;
    unsigned scale;
  };
  static __device__ __forceinline__ void arrived(Raw& r) {
    asm volatile("" : "+v"(r.codes), "+v"(r.scale));
  }
  const uint8_t* codes;
  const uint8_t* scales;
  __device__ __forceinline__ Raw load(size_t at) const {
    return Raw{*(const mx8::u32x2*)(codes + at), scales[at / 32]};
  }
  static __device__ __forceinline__ void values(const Raw& r, float* v) {
    mx8::decode(r.codes, r.scale, v);
  }
};

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

// Whether piece p of a thread lies in the row.
__device__ __forceinline__ bool inside(int p, int H) {
  return (p * (int)blockDim.x + (int)threadIdx.x) * 8 < H;
}

// Rows whose sums leave fp32's range, as inv_rms has them.
__device__ __forceinline__ bool too_large(float ss) { return !(ss < __builtin_inff()); }
__device__ __forceinline__ bool too_small(float ss, float eps) {
  return ss < 0x1p-90f && eps < 0x1p-100f;
}

// v = v - mean(v), and the sum of its squares: part of 2 sums.
template <int P>
__device__ __forceinline__ float deviations(float (&v)[P][8], int H, float (*part)[kMaxWaves]) {
  float s[1] = {0.0f};
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (inside(p, H))
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += v[p][i];
  row_sums<kMaxWaves>(s, part);
  const float m = s[0] / (float)H;
  s[0] = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (inside(p, H))
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[p][i] -= m;
        s[0] = fmaf(v[p][i], v[p][i], s[0]);
      }
  row_sums<kMaxWaves>(s, part + 1);
  return s[0];
}

// MEAN: by mean and variance; else y is that of norm_kernel, bit for bit.
// SAVE: x in 8 bits to codes and scales (a row's pieces of 4 neighbouring
// threads are a block of 32).
template <typename T, typename U, int P, bool MEAN, bool SAVE>
__global__ __launch_bounds__(kMaxThreads) void norm_save_kernel(
    const T* x, const float* __restrict__ w, const float* __restrict__ b, float eps, int rows,
    int H, U* y, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ float part[4][kMaxWaves];
  const bool one_wave = blockDim.x == kWave;
  const unsigned t = row_of_thread();
  if (t >= (unsigned)rows) return;   // a whole wave, and then blocks have no barrier
  if (MEAN && !one_wave) {
    if (threadIdx.x < 4 * kMaxWaves) part[threadIdx.x / kMaxWaves][threadIdx.x % kMaxWaves] = 0.0f;
    lds_barrier();
  }
  float v[P][8];
  float ss = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      const size_t at = (size_t)t * H + h;
      Row8<T>::load(x + at, v[p]);
      if (SAVE) {
        unsigned byte;
        *(mx8::u32x2*)(codes + at) = mx8::encode(v[p], byte);
        if ((threadIdx.x & 3) == 0) scales[at / 32] = (uint8_t)byte;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(v[p][i], v[p][i], ss);
    }
  }
  float r;
  if (MEAN) {
    ss = deviations(v, H, part);
    float f = 1.0f;
    if (too_large(ss)) {
      // the deviations may be lost too: the values again, scaled
      f = 0x1p-96f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int h = (p * blockDim.x + threadIdx.x) * 8;
        if (h < H) {
          Row8<T>::load(x + (size_t)t * H + h, v[p]);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[p][i] *= f;
        }
      }
      ss = deviations(v, H, part + 2);
    } else if (too_small(ss, eps)) {
      f = 0x1p96f;
      float s[1] = {0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (inside(p, H))
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[p][i] *= f;
            s[0] = fmaf(v[p][i], v[p][i], s[0]);
          }
      row_sums<kMaxWaves>(s, part + 2);
      ss = s[0];
    }
    r = rsqrtf(ss / (float)H + eps * f * f);
  } else {
    r = inv_rms(v, ss, eps, H, part, one_wave);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = (p * blockDim.x + threadIdx.x) * 8;
    if (h < H) {
      float g[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (w) Row8<float>::load(w + h, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = v[p][i] * r * g[i];
      if (MEAN && b) {
        Row8<float>::load(b + h, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] += g[i];
      }
      Row8<U>::store(y + (size_t)t * H + h, v[p]);
    }
  }
}

// A block goes over the rows blockIdx.x * blockDim.y + threadIdx.y, and so on;
// a row has THREADS threads at most, of P pieces each.  sum_w, sum_b: the
// block's sums over its rows go to row blockIdx.x of them, `stride` floats a
// row; NULL: not asked for.
// Up to 8192 values a row has at most 256 threads, with the weight in registers
// and the next row's x and dy in flight while one is worked on: what a row costs
// once (its sums, addresses) is shared by up to 32 values a lane, and two or
// three blocks of a CU wait for different things.  Longer rows have neither.
template <typename DY, typename X, typename DX, int P, int THREADS, bool MEAN>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(
    Source<DY> dy, Source<X> x, const float* __restrict__ w, float eps, int rows, int H,
    Source<DX> d_residual, DX* dx, float* __restrict__ sum_w, float* __restrict__ sum_b,
    int stride) {
  constexpr bool kAhead = THREADS <= 256;
  constexpr int kSums = 9, kWaves = THREADS / kWave < 16 ? 4 : 16;
  // the sums of one row are read while those of the next are written
  __shared__ __attribute__((aligned(16))) float part[2][kSums][kWaves];
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 2 * kSums * kWaves;
       i += blockDim.x * blockDim.y)
    (&part[0][0][0])[i] = 0.0f;
  __syncthreads();
  const long long step = (long long)gridDim.x * blockDim.y;
  long long t = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  // Only a thread's last piece may lie behind the row (the shape sees to it).
  // Loads are made for all pieces, from the row's start for one that is behind
  // and from the last row for one that is no more: a load under a condition
  // would be waited for where it is made, to be merged with what was there.
  const bool last_in = inside(P - 1, H);
  const float inv_h = 1.0f / (float)H;
  int at[P];
  float dw[P][8] = {}, db[P][8] = {}, weight[kAhead ? P : 1][8];
#pragma unroll
  for (int p = 0; p < P; ++p)
    at[p] = p < P - 1 || last_in ? (p * (int)blockDim.x + (int)threadIdx.x) * 8 : 0;
  const auto weights = [&](int p, float (&g)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.0f;
    if (w) Row8<float>::load(w + at[p], g);
  };
  typename Source<DY>::Raw next_dy[P];
  typename Source<X>::Raw next_x[P];
  const auto fetch = [&](long long row) {
    const size_t start = (size_t)min(row, (long long)rows - 1) * H;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      next_x[p] = x.load(start + at[p]);
      next_dy[p] = dy.load(start + at[p]);
    }
  };
  if (kAhead) {
#pragma unroll
    for (int p = 0; p < P; ++p) weights(p, weight[p]);
    fetch(t);
  }
  for (int turn = 0; t < rows; t += step, turn ^= 1) {
    const size_t row = (size_t)t * H;
    float v[P][8], d[P][8];   // x, then its deviations; dy
    typename Source<DX>::Raw res[P];
    if (!kAhead) fetch(t);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      Source<X>::arrived(next_x[p]);
      Source<DY>::arrived(next_dy[p]);
      Source<X>::values(next_x[p], v[p]);
      Source<DY>::values(next_dy[p], d[p]);
    }
    if (d_residual.p) {
#pragma unroll
      for (int p = 0; p < P; ++p) res[p] = d_residual.load(row + at[p]);
    }
    if (kAhead) fetch(t + step);
    // behind the row: nothing to any sum
    const auto clear_behind = [&](float (&a)[P][8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[P - 1][i] = last_in ? a[P - 1][i] : 0.0f;
    };
    clear_behind(v);
    clear_behind(d);
    float s[3];
    // v = v - mean(v)
    const auto center = [&](float (*lds)[kWaves]) {
      if (!MEAN) return;
      float a[1] = {0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) a[0] += v[p][i];
      row_sums<kWaves>(a, lds);
      const float m = a[0] * inv_h;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] -= m;
      clear_behind(v);
    };
    // the squares of v, g times v, and g
    const auto sums = [&](float (*lds)[kWaves]) {
      s[0] = s[1] = s[2] = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float g[8];
        if (!kAhead) weights(p, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gi = d[p][i] * (kAhead ? weight[p][i] : g[i]);
          s[0] = fmaf(v[p][i], v[p][i], s[0]);
          s[1] = fmaf(gi, v[p][i], s[1]);
          if (MEAN) s[2] += gi;
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
    center(part[turn]);
    sums(part[turn] + 1);
    // n = v to_n, dx = (..) root f
    float f = 1.0f, root = rsqrtf(s[0] * inv_h + eps), to_n = root;
    if (too_large(s[0]) || too_small(s[0], eps) || !(fabsf(s[1]) < __builtin_inff())) {
      // rare, and the same for the row's threads: v scaled, then normed before it meets g
      const bool large = too_large(s[0]);
      f = large ? 0x1p-96f : too_small(s[0], eps) ? 0x1p96f : 1.0f;
      float a[1] = {0.0f};
      if (large) {   // the deviations may be lost already
#pragma unroll
        for (int p = 0; p < P; ++p) Source<X>::values(x.load(row + at[p]), v[p]);
        clear_behind(v);
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] *= f;
      if (large) center(part[turn] + 4);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) a[0] = fmaf(v[p][i], v[p][i], a[0]);
      row_sums<kWaves>(a, part[turn] + 5);
      root = rsqrtf(a[0] * inv_h + eps * f * f);
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[p][i] *= root;
      to_n = 1.0f;
      sums(part[turn] + 6);
    }
    const float c = to_n * s[1] * inv_h, mean_g = MEAN ? s[2] * inv_h : 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float g[8], o[8] = {};
      if (!kAhead) weights(p, g);
      if (d_residual.p) Source<DX>::values(res[p], o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = v[p][i] * to_n, gi = d[p][i] * (kAhead ? weight[p][i] : g[i]);
        o[i] = fmaf((gi - mean_g - n * c) * root, f, o[i]);   // root f may pass 2^128
        dw[p][i] = fmaf(d[p][i], n, dw[p][i]);
        db[p][i] += d[p][i];
      }
      if (p < P - 1 || last_in) Row8<DX>::store(dx + row + at[p], o);
    }
  }
  if (!sum_w && !sum_b) return;
  if (P == 1 && kAhead && blockDim.y > 1) {
    // the block's rows at a time share a column: joined in their order
    __shared__ float other[3][2][kWave * 8];
    if (threadIdx.y > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        other[threadIdx.y - 1][0][i * kWave + threadIdx.x] = dw[0][i];
        other[threadIdx.y - 1][1][i * kWave + threadIdx.x] = db[0][i];
      }
    }
    __syncthreads();
    if (threadIdx.y > 0) return;
    for (int y = 1; y < (int)blockDim.y; ++y)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dw[0][i] += other[y - 1][0][i * kWave + threadIdx.x];
        db[0][i] += other[y - 1][1][i * kWave + threadIdx.x];
      }
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
    if (p < P - 1 || last_in) {
      const size_t to = (size_t)blockIdx.x * stride + at[p];
      if (sum_w) Row8<float>::store(sum_w + to, dw[p]);
      if (MEAN && sum_b) Row8<float>::store(sum_b + to, db[p]);
    }
}

// d[h] = sum over n rows of sums[.][h], 64 columns a block; blockIdx.y: the
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

// The backward pass's blocks: four rows of a wave each, or a row of a block.
Shape backward_shape(int T, int H) {
  Shape s;
  s.P = std::min(ceil_div(H, 2048), 4u);
  const int per = ceil_div(ceil_div(H, 8 * s.P), kWave) * kWave;
  const int rows = per == kWave ? 4 : 1;
  s.block = dim3(per, rows);
  // blocks for two waves a SIMD, each with a few rows
  const unsigned most = 256 * std::max(1, 512 / (per * rows));
  s.grid = dim3(std::min(ceil_div(T, rows), most));
  return s;
}

}  // namespace

size_t norm_backward_ws_bytes(int T, int H) {
  return (size_t)backward_shape(T, H).grid.x * 2 * H * sizeof(float);
}

namespace {

template <typename T, typename U>
void save_t(bool mean, const void* x, const float* w, const float* b, float eps, int T_, int H,
            void* y, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const Shape s = shape(T_, H);
#define MOE_NORM(P, MEAN, SAVE)                                                               \
  MOE_LAUNCH(MEAN ? "layer_norm" : "norm_checkpoint", st,                                     \
             norm_save_kernel<T, U, P, MEAN, SAVE><<<s.grid, s.block, 0, st>>>(               \
                 (const T*)x, w, b, eps, T_, H, (U*)y, codes, scales))
#define MOE_NORM_P(MEAN, SAVE) \
  if (s.P == 1)                \
    MOE_NORM(1, MEAN, SAVE);   \
  else if (s.P == 2)           \
    MOE_NORM(2, MEAN, SAVE);   \
  else                         \
    MOE_NORM(4, MEAN, SAVE);
  if (!mean) {
    MOE_NORM_P(false, true)
  } else if (codes) {
    MOE_NORM_P(true, true)
  } else {
    MOE_NORM_P(true, false)
  }
#undef MOE_NORM_P
#undef MOE_NORM
}

template <typename DY, typename X, typename DX>
void backward_t(bool mean, const void* dy, Source<X> x, const float* w, float eps, int T, int H,
                const void* d_residual, void* dx, float* d_weight, float* d_bias, float* ws,
                hipStream_t st) {
  const Shape s = backward_shape(T, H);
  // one block has the whole sums
  const bool join = s.grid.x > 1 && (d_weight || d_bias);
  float* sum_w = join ? ws : d_weight;
  float* sum_b = join ? ws + H : d_bias;
#define MOE_NORM(P, THREADS, MEAN)                                                           \
  MOE_LAUNCH("norm_backward", st,                                                            \
             norm_backward_kernel<DY, X, DX, P, THREADS, MEAN><<<s.grid, s.block, 0, st>>>(  \
                 Source<DY>{(const DY*)dy}, x, w, eps, T, H, Source<DX>{(const DX*)d_residual}, \
                 (DX*)dx, sum_w, sum_b, 2 * H))
#define MOE_NORM_P(MEAN)         \
  if (H > 8192)                  \
    MOE_NORM(4, 1024, MEAN);     \
  else if (s.P == 1)             \
    MOE_NORM(1, 256, MEAN);      \
  else if (s.P == 2)             \
    MOE_NORM(2, 256, MEAN);      \
  else if (s.P == 3)             \
    MOE_NORM(3, 256, MEAN);      \
  else                           \
    MOE_NORM(4, 256, MEAN);
  if (mean) {
    MOE_NORM_P(true)
  } else {
    MOE_NORM_P(false)
  }
#undef MOE_NORM_P
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
  if (x_scales)
    backward_t<DY, Mx8, DX>(mean, dy, Source<Mx8>{(const uint8_t*)x, x_scales}, w, eps, T, H,
                            d_residual, dx, d_weight, d_bias, ws, st);
  else if (x_dtype == MOE_BF16)
    backward_t<DY, bf16, DX>(mean, dy, Source<bf16>{(const bf16*)x}, w, eps, T, H, d_residual, dx,
                             d_weight, d_bias, ws, st);
  else
    backward_t<DY, float, DX>(mean, dy, Source<float>{(const float*)x}, w, eps, T, H, d_residual,
                              dx, d_weight, d_bias, ws, st);
}

}  // namespace

hipError_t launch_norm_save(bool mean, const void* x, int x_dtype, const float* weight,
                            const float* bias, float eps, int T, int H, void* y, int y_dtype,
                            uint8_t* codes, uint8_t* scales, hipStream_t s) {
#define MOE_SAVE(T_, U) save_t<T_, U>(mean, x, weight, bias, eps, T, H, y, codes, scales, s)
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

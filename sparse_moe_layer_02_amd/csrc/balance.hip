// The losses of a batch's routing and the gradient of the router's logits.
//   load[s][e] = E counts[s][e] / (K tokens[s]), averaged over e's group
//   balance = 1/N sum over t, e of load[seq[t]][e] p[t][e],  z = 1/N sum of lse^2
//   d_logits = p (g - sum p g + z's term)
// The picks are counted first (integers: exact in any order).  The balance loss
// is then one sweep over the logits: each row's probabilities times its
// sequence's loads, so that no sum over tokens is held for every expert of
// every sequence.  The gradient is one sweep too, a row in registers between
// its read and its write.  A wave has a row: lane l the experts l + 64 i.
#include "train_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxRowBlocks = 2048;

// Sequence of a token, or -1 for padding.
__device__ __forceinline__ int sequence(const int32_t* seq, int n_seq, long long t) {
  if (!seq) return 0;
  const int s = seq[t];
  return s >= 0 && s < n_seq ? s : -1;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = kWave / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

__global__ __launch_bounds__(kThreads) void balance_clear(int32_t* counts, long long n,
                                                          int32_t* tokens, int n_tokens) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) counts[i] = 0;
  if (i < n_tokens) tokens[i] = 0;
}

// A block counts the picks of kCountTokens tokens: those of the first one's
// sequence, as a rule all of them, in LDS, the others in memory.
constexpr int kCountThreads = 1024;
constexpr int kCountTokens = 512;
__global__ __launch_bounds__(kCountThreads) void balance_count(
    const int32_t* __restrict__ idx, const int32_t* __restrict__ seq, int n_seq, int T, int E,
    int K, int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  __shared__ int hist[kMaxRouteE];
  __shared__ int mine;
  const int t0 = blockIdx.x * kCountTokens, n = min(kCountTokens, T - t0);
  const int home = sequence(seq, n_seq, t0);
  for (int e = threadIdx.x; e < E; e += kCountThreads) hist[e] = 0;
  if (threadIdx.x == 0) mine = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n * K; i += kCountThreads) {
    const int e = idx[(size_t)t0 * K + i], s = sequence(seq, n_seq, t0 + i / K);
    if (e < 0 || e >= E || s < 0) continue;
    if (s == home)
      atomicAdd(&hist[e], 1);
    else
      atomicAdd(&counts[(size_t)s * E + e], 1);
  }
  if (threadIdx.x < n) {
    const int s = sequence(seq, n_seq, t0 + threadIdx.x);
    if (s >= 0) {
      if (s == home)
        atomicAdd(&mine, 1);
      else
        atomicAdd(&tokens[s], 1);
    }
  }
  __syncthreads();
  if (home < 0) return;
  for (int e = threadIdx.x; e < E; e += kCountThreads)
    if (hist[e]) atomicAdd(&counts[(size_t)home * E + e], hist[e]);
  if (threadIdx.x == 0 && mine) atomicAdd(&tokens[home], mine);
}

// A sequence's loads.
__global__ __launch_bounds__(kThreads) void balance_load(const int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ tokens, int n_seq,
                                                         const int32_t* __restrict__ group, int E,
                                                         int K, float* __restrict__ load) {
  __shared__ int sum[kMaxRouteE], size[kMaxRouteE];
  const int s = blockIdx.x;
  const int n = tokens[s];
  if (s == 0) {   // all tokens
    __shared__ int all;
    if (threadIdx.x == 0) all = 0;
    __syncthreads();
    int mine = 0;
    for (int i = threadIdx.x; i < n_seq; i += kThreads) mine += tokens[i];
    atomicAdd(&all, mine);
    __syncthreads();
    if (threadIdx.x == 0) tokens[n_seq] = all;
  }
  if (group) {
    for (int e = threadIdx.x; e < E; e += kThreads) sum[e] = size[e] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
      const int g = group[e];
      if (g >= 0 && g < E) {
        atomicAdd(&sum[g], counts[(size_t)s * E + e]);
        atomicAdd(&size[g], 1);
      }
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e < E; e += kThreads) {
    float v = 0.0f;
    if (n > 0) {
      const double even = (double)E / ((double)K * n);
      const int g = group ? group[e] : e;
      if (!group)
        v = (float)(even * counts[(size_t)s * E + e]);
      else if (g >= 0 && g < E)
        v = (float)(even * sum[g] / size[g]);
    }
    load[(size_t)s * E + e] = v;
  }
}

// A row's probabilities (p, times 1 / the sum) and the logarithm of its sum.
// A row of -inf alone has zeros.
template <int EPL>
struct Softmax {
  float p[EPL];
  float lse;
  __device__ __forceinline__ void row(const float* l, int E, int lane) {
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + kWave * i;
      p[i] = e < E ? l[e] : -INFINITY;
      top = fmaxf(top, p[i]);
    }
    top = wave_max(top);
    // a NaN is no maximum, but leaves none of the sum
    const float shift = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = expf(p[i] - shift);
      sum += p[i];
    }
    sum = wave_sum(sum);
    lse = sum == 0.0f ? 0.0f : shift + logf(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] *= inv;
  }
};

// Per block: the sums over its rows of load p and of lse^2.
template <int EPL>
__global__ __launch_bounds__(kThreads) void balance_rows(const float* __restrict__ logits,
                                                         const int32_t* __restrict__ seq,
                                                         int n_seq, int T, int E,
                                                         const float* __restrict__ load,
                                                         double* __restrict__ sums) {
  __shared__ double part[2][kWaves];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  double balance = 0.0, z = 0.0;
  for (long long t = (long long)blockIdx.x * kWaves + wave; t < T;
       t += (long long)gridDim.x * kWaves) {
    const int s = sequence(seq, n_seq, t);
    if (s < 0) continue;
    Softmax<EPL> m;
    m.row(logits + t * E, E, lane);
    const float* f = load + (size_t)s * E;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + kWave * i < E) dot = fmaf(m.p[i], f[lane + kWave * i], dot);
    balance += wave_sum(dot);
    z += (double)m.lse * m.lse;
  }
  if (lane == 0) {
    part[0][wave] = balance;
    part[1][wave] = z;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    double v = 0.0;
    for (int w = 0; w < kWaves; ++w) v += part[threadIdx.x][w];
    sums[(size_t)blockIdx.x * 2 + threadIdx.x] = v;
  }
}

// losses from n blocks' sums.
__global__ __launch_bounds__(kThreads) void balance_finish(const double* __restrict__ sums, int n,
                                                           const int32_t* __restrict__ tokens,
                                                           int n_seq, float balance_coef,
                                                           float z_coef,
                                                           float* __restrict__ losses) {
  __shared__ double part[2][kThreads];
  double a = 0.0, b = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    a += sums[2 * i];
    b += sums[2 * i + 1];
  }
  part[0][threadIdx.x] = a;
  part[1][threadIdx.x] = b;
  __syncthreads();
  for (int off = kThreads / 2; off > 0; off >>= 1) {
    if (threadIdx.x < off) {
      part[0][threadIdx.x] += part[0][threadIdx.x + off];
      part[1][threadIdx.x] += part[1][threadIdx.x + off];
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int all = tokens[n_seq];
    losses[0] = all > 0 ? (float)(balance_coef * part[0][0] / all) : 0.0f;
    losses[1] = all > 0 ? (float)(z_coef * part[1][0] / all) : 0.0f;
  }
}

// d_logits may be logits: a wave has read the row that it overwrites.
template <int EPL>
__global__ __launch_bounds__(kThreads) void route_backward(
    const float* logits, const int32_t* __restrict__ idx, const float* __restrict__ d_gate,
    const int32_t* __restrict__ seq, int n_seq, const int32_t* __restrict__ tokens,
    const float* __restrict__ load, const float* __restrict__ d_losses, float balance_coef,
    float z_coef, int T, int E, int K, float* d_logits) {
  __shared__ float gates[kWaves][kWave * EPL];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  float* mine = gates[wave];
  if (d_gate) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) mine[lane + kWave * i] = 0.0f;
  }
  float cb = 0.0f, cz = 0.0f;
  if (load) {
    const int all = tokens[n_seq];
    if (all > 0) {
      cb = balance_coef * (d_losses ? d_losses[0] : 1.0f) / (float)all;
      cz = 2.0f * z_coef * (d_losses ? d_losses[1] : 1.0f) / (float)all;
    }
  }
  for (long long t = (long long)blockIdx.x * kWaves + wave; t < T;
       t += (long long)gridDim.x * kWaves) {
    Softmax<EPL> m;
    m.row(logits + t * E, E, lane);
    float g[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) g[i] = 0.0f;
    if (d_gate) {
      // the picks one after the other: equal ones add up in their order
      for (int k0 = 0; k0 < K; k0 += kWave) {
        const int k = k0 + lane;
        const int e = k < K ? idx[t * K + k] : -1;
        const float d = k < K ? d_gate[t * K + k] : 0.0f;
        for (int j = 0; j < min(kWave, K - k0); ++j) {
          if (lane == j && e >= 0 && e < E) mine[e] += d;
          wave_lds_sync();
        }
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        g[i] = mine[lane + kWave * i];
        mine[lane + kWave * i] = 0.0f;
      }
      wave_lds_sync();
    }
    float more = 0.0f;
    if (load) {
      const int s = sequence(seq, n_seq, t);
      if (s >= 0) {
        const float* f = load + (size_t)s * E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (lane + kWave * i < E) g[i] = fmaf(cb, f[lane + kWave * i], g[i]);
        more = cz * m.lse;
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (m.p[i] == 0.0f) g[i] = 0.0f;   // a masked pick's gradient may be anything
      dot = fmaf(m.p[i], g[i], dot);
    }
    dot = wave_sum(dot);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + kWave * i < E) d_logits[t * E + lane + kWave * i] = m.p[i] * (g[i] - dot + more);
  }
}

unsigned row_blocks(int T) { return min(ceil_div(T, kWaves), (unsigned)kMaxRowBlocks); }

}  // namespace

size_t balance_ws_bytes(int T, int E, int n_seq) {
  (void)E;
  (void)n_seq;
  return (size_t)row_blocks(T) * 2 * sizeof(double);
}

#define MOE_BY_WIDTH(E, CALL)             \
  do {                                    \
    const int epl = ((E) + kWave - 1) / kWave; \
    if (epl <= 1) CALL(1);                \
    else if (epl <= 2) CALL(2);           \
    else if (epl <= 4) CALL(4);           \
    else if (epl <= 8) CALL(8);           \
    else if (epl <= 12) CALL(12);         \
    else CALL(16);                        \
  } while (0)

hipError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* seq,
                               int n_seq, const int32_t* group, int T, int E, int K,
                               float balance_coef, float z_coef, int32_t* counts, int32_t* tokens,
                               float* load, float* losses, void* ws, hipStream_t s) {
  const long long n = (long long)n_seq * E;
  double* sums = (double*)ws;
  const unsigned blocks = row_blocks(T);
  MOE_LAUNCH("balance_clear", s,
             balance_clear<<<ceil_div((size_t)max(n, (long long)n_seq + 1), kThreads), kThreads, 0,
                             s>>>(counts, n, tokens, n_seq + 1));
  MOE_LAUNCH("balance_count", s,
             balance_count<<<ceil_div(T, kCountTokens), kCountThreads, 0, s>>>(
                 idx, seq, n_seq, T, E, K, counts, tokens));
  MOE_LAUNCH("balance_load", s,
             balance_load<<<n_seq, kThreads, 0, s>>>(counts, tokens, n_seq, group, E, K, load));
#define MOE_BALANCE(EPL)                                                                    \
  MOE_LAUNCH("balance_rows", s,                                                             \
             balance_rows<EPL><<<blocks, kThreads, 0, s>>>(logits, seq, n_seq, T, E, load, sums))
  MOE_BY_WIDTH(E, MOE_BALANCE);
#undef MOE_BALANCE
  MOE_LAUNCH("balance_finish", s,
             balance_finish<<<1, kThreads, 0, s>>>(sums, blocks, tokens, n_seq, balance_coef,
                                                   z_coef, losses));
  return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, const int32_t* idx, const float* d_gate,
                                 const int32_t* seq, int n_seq, const int32_t* tokens,
                                 const float* load, const float* d_losses, float balance_coef,
                                 float z_coef, int T, int E, int K, float* d_logits,
                                 hipStream_t s) {
#define MOE_BACKWARD(EPL)                                                                   \
  MOE_LAUNCH("route_backward", s,                                                           \
             route_backward<EPL><<<row_blocks(T), kThreads, 0, s>>>(                        \
                 logits, idx, d_gate, seq, n_seq, tokens, load, d_losses, balance_coef,     \
                 z_coef, T, E, K, d_logits))
  MOE_BY_WIDTH(E, MOE_BACKWARD);
#undef MOE_BACKWARD
  return hipGetLastError();
}

}  // namespace moe

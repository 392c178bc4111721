// The losses of a batch's routing and the gradient of the router's logits.
//   load[s][e] = E counts[s][e] / (K tokens[s]), averaged over e's group
//   balance = 1/N sum over t, e of load[seq[t]][e] p[t][e],  z = 1/N sum of lse^2
//   d_logits = p (g - sum p g + z's term)
// The picks are counted first (integers: exact in any order).  The balance loss
// is then one sweep over the logits: each row's probabilities times its
// sequence's loads, so that no sum over tokens is held for every expert of
// every sequence.  The gradient is one sweep too, a row in registers between
// its read and its write.  Rows belong to groups of 8 to 64 lanes, by the
// pool's size, so that a wave has work for its lanes on small pools too.
#include <algorithm>

#include "train_internal.h"
#include "wave.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kCountThreads = 1024;   // at least kMaxRouteE: an expert a thread
constexpr int kLossThreads = 1024;
constexpr unsigned kLossBlocks = 256, kGradientBlocks = 2048;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// Sequence of a token, or -1 for padding.
__device__ __forceinline__ int sequence(const int32_t* seq, int n_seq, long long t) {
  if (!seq) return 0;
  const int s = seq[t];
  return s >= 0 && s < n_seq ? s : -1;
}

// ------------------------------------------------------- counts and loads --

// The loads of sequence s by a block of at least E threads: thread e has the
// expert's picks and group, n tokens.  sum, size: LDS for the groups.
__device__ __forceinline__ void loads_of(int s, int picks, int g, bool grouped, int n, int E, int K,
                                         int* sum, int* size, float* load) {
  const int e = threadIdx.x;
  const bool in = e < E && g >= 0 && g < E;
  if (grouped) {
    if (e < E) sum[e] = size[e] = 0;
    __syncthreads();
    if (in) {
      atomicAdd(&sum[g], picks);
      atomicAdd(&size[g], 1);
    }
    __syncthreads();
  }
  if (e >= E) return;
  const double even = n > 0 ? (double)E / ((double)K * n) : 0.0;
  float v = 0.0f;
  if (!grouped)
    v = (float)(even * picks);
  else if (in)
    v = (float)(even * sum[g] / size[g]);
  load[(size_t)s * E + e] = v;
}

// Counts and loads of sequence s by a block, which looks at all tokens'
// sequences, 64 tokens to a wave, and counts the picks of those of its own in LDS.
constexpr int kPicks = 12;  // picks that a lane has in flight (2730 x 768, K 12: 15.9 us the
                            // losses so, 19.6 with one, 16.5 with 4, 17.5 with 24)
struct CountLds {
  int hist[kMaxRouteE], sum[kMaxRouteE], size[kMaxRouteE];
  int mine, all;
};
__device__ __forceinline__ void count_sequence(int s, CountLds& lds, const int32_t* idx,
                                               const int32_t* seq, int n_seq,
                                               const int32_t* group, int T, int E, int K,
                                               int32_t* counts, int32_t* tokens, float* load) {
  const int lane = threadIdx.x & (kWave - 1), expert = threadIdx.x;
  const int g = group && expert < E ? group[expert] : expert;
  lds.hist[expert] = 0;
  if (threadIdx.x == 0) lds.mine = lds.all = 0;
  __syncthreads();
  int n = 0, inside = 0;
  for (int t0 = threadIdx.x / kWave * kWave; t0 < T; t0 += kCountThreads) {
    const int q = t0 + lane < T ? sequence(seq, n_seq, t0 + lane) : -1;
    const uint64_t here = __ballot(q == s);
    inside += __popcll(__ballot(q >= 0));
    n += __popcll(here);
    if (here == 0) continue;
    const int32_t* picks = idx + (size_t)t0 * K;
    // bits of tokens past T are not set: their picks are not read
    for (int i0 = lane; i0 < kWave * K; i0 += kPicks * kWave) {
      int e[kPicks];
#pragma unroll
      for (int k = 0; k < kPicks; ++k) {
        const int i = i0 + k * kWave;
        e[k] = i < kWave * K && (here >> (i / K) & 1) ? picks[i] : -1;
      }
#pragma unroll
      for (int k = 0; k < kPicks; ++k)
        if (e[k] >= 0 && e[k] < E) atomicAdd(&lds.hist[e[k]], 1);
    }
  }
  if (lane == 0) {
    atomicAdd(&lds.mine, n);
    atomicAdd(&lds.all, inside);
  }
  __syncthreads();
  if (expert < E) counts[(size_t)s * E + expert] = lds.hist[expert];
  if (threadIdx.x == 0) {
    tokens[s] = lds.mine;
    if (s == 0) tokens[n_seq] = lds.all;
  }
  loads_of(s, lds.hist[expert], g, group != nullptr, lds.mine, E, K, lds.sum, lds.size, load);
}

__global__ __launch_bounds__(kCountThreads) void balance_count_sequence(
    const int32_t* __restrict__ idx, const int32_t* __restrict__ seq, int n_seq,
    const int32_t* __restrict__ group, int T, int E, int K, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, float* __restrict__ load, unsigned* __restrict__ ticket) {
  __shared__ CountLds lds;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
  count_sequence(blockIdx.x, lds, idx, seq, n_seq, group, T, E, K, counts, tokens, load);
}

__global__ __launch_bounds__(kThreads) void balance_clear(int32_t* counts, long long n,
                                                          int32_t* tokens, int n_tokens,
                                                          unsigned* ticket) {
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) counts[i] = 0;
  if (i < n_tokens) tokens[i] = 0;
  if (i == 0) *ticket = 0;
}

// A block counts the picks of kCountTokens tokens at a time: those of the first
// one's sequence, as a rule all of them, in LDS, the others in memory.
constexpr int kCountTokens = 256;
constexpr unsigned kCountBlocks = 4096;
__global__ __launch_bounds__(kCountThreads) void balance_count(
    const int32_t* __restrict__ idx, const int32_t* __restrict__ seq, int n_seq, int T, int E,
    int K, int32_t* __restrict__ counts, int32_t* __restrict__ tokens) {
  __shared__ int hist[kMaxRouteE];
  __shared__ int mine, all;
  for (long long t0 = (long long)blockIdx.x * kCountTokens; t0 < T;
       t0 += (long long)gridDim.x * kCountTokens) {
    const int n = (int)min((long long)kCountTokens, T - t0);
    const int home = sequence(seq, n_seq, t0);
    for (int e = threadIdx.x; e < E; e += kCountThreads) hist[e] = 0;
    if (threadIdx.x == 0) mine = all = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < n * K; i += kCountThreads) {
      const int e = idx[t0 * K + i], s = sequence(seq, n_seq, t0 + i / K);
      if (e < 0 || e >= E || s < 0) continue;
      if (s == home)
        atomicAdd(&hist[e], 1);
      else
        atomicAdd(&counts[(size_t)s * E + e], 1);
    }
    if (threadIdx.x < n) {
      const int s = sequence(seq, n_seq, t0 + threadIdx.x);
      if (s >= 0) {
        atomicAdd(&all, 1);
        if (s == home)
          atomicAdd(&mine, 1);
        else
          atomicAdd(&tokens[s], 1);
      }
    }
    __syncthreads();
    if (home >= 0)
      for (int e = threadIdx.x; e < E; e += kCountThreads)
        if (hist[e]) atomicAdd(&counts[(size_t)home * E + e], hist[e]);
    if (threadIdx.x == 0) {
      if (all) atomicAdd(&tokens[n_seq], all);
      if (mine) atomicAdd(&tokens[home], mine);
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kCountThreads) void balance_load(const int32_t* __restrict__ counts,
                                                         const int32_t* __restrict__ tokens,
                                                         const int32_t* __restrict__ group, int E,
                                                         int K, float* __restrict__ load) {
  __shared__ int sum[kMaxRouteE], size[kMaxRouteE];
  const int s = blockIdx.x, e = threadIdx.x;
  loads_of(s, e < E ? counts[(size_t)s * E + e] : 0, group && e < E ? group[e] : e,
           group != nullptr, tokens[s], E, K, sum, size, load);
}

// ------------------------------------------------------------------ rows --

// A row of E values in the registers of W lanes: N pieces of VEC a lane, piece
// i of lane l at (i W + l) VEC.
template <int W, int N, int VEC>
struct RowOf {
  static constexpr int kSize = W * N * VEC;
  static __device__ __forceinline__ int at(int i, int l) { return (i * W + l) * VEC; }

  static __device__ __forceinline__ void load(const float* p, int E, int l, float (&v)[N][VEC],
                                              float behind) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = behind;
      if (at(i, l) < E) {   // VEC divides E
        if (VEC == 4)
          *(f32x4*)v[i] = *(const f32x4*)(p + at(i, l));
        else
          v[i][0] = p[at(i, l)];
      }
    }
  }
  // Past the caches (16384 x 768: 17.7 us the gradient's pass, 22.4 with the default
  // policy; loads past them 23.4).
  static __device__ __forceinline__ void store(float* p, int E, int l, const float (&v)[N][VEC]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i, l) < E) {
        if (VEC == 4)
          __builtin_nontemporal_store(*(const f32x4*)v[i], (f32x4*)(p + at(i, l)));
        else
          __builtin_nontemporal_store(v[i][0], p + at(i, l));
      }
  }

  // Logits to probabilities; returns the logarithm of their sum.  A row of -inf
  // alone gives zeros.  exp is 2^x of a product rounded once: off by the
  // distance from the largest logit times half a step, beside the sum's own
  // rounding.
  static __device__ __forceinline__ float softmax(float (&p)[N][VEC]) {
    float top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) top = fmaxf(top, p[i][j]);
    top = group_max<W>(top);
    if (top == -INFINITY) top = 0.0f;   // (a NaN is no maximum, but leaves none of the sum)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        p[i][j] = __builtin_amdgcn_exp2f((p[i][j] - top) * kLog2e);
        sum += p[i][j];
      }
    sum = group_sum<W>(sum);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) p[i][j] *= inv;
    return sum == 0.0f ? 0.0f : fmaf(__builtin_amdgcn_logf(sum), kLn2, top);
  }
};

// Sums of load p and of lse^2 over the rows first, first + step, ..., in the
// first lanes of the rows' groups.
template <int W, int N, int VEC>
__device__ __forceinline__ void loss_rows(const float* logits, const int32_t* seq, int n_seq,
                                          int T, int E, const float* load, long long first,
                                          long long step, double (&v)[2]) {
  typedef RowOf<W, N, VEC> Row;
  const int l = threadIdx.x % W;
  v[0] = v[1] = 0.0;
  for (long long t = first; t < T; t += step) {
    const int s = sequence(seq, n_seq, t);
    if (s < 0) continue;
    float p[N][VEC], f[N][VEC];
    Row::load(logits + t * E, E, l, p, -INFINITY);
    Row::load(load + (size_t)s * E, E, l, f, 0.0f);
    const float lse = Row::softmax(p);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) dot = fmaf(p[i][j], f[i][j], dot);
    dot = group_sum<W>(dot);
    if (l == 0) {
      v[0] += dot;
      v[1] += (double)lse * lse;
    }
  }
}

// The waves' sums, then the block's, in thread 0.
__device__ __forceinline__ void join_losses(double (&v)[2], double (*part)[kLossThreads / kWave]) {
  constexpr int kWaves = kLossThreads / kWave;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1) v[k] += __shfl_xor(v[k], off);
    if ((threadIdx.x & (kWave - 1)) == 0) part[k][threadIdx.x / kWave] = v[k];
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int k = 0; k < 2; ++k) {
      v[k] = 0.0;
      for (int w = 0; w < kWaves; ++w) v[k] += part[k][w];
    }
}

__device__ __forceinline__ void write_losses(const double (&v)[2], int all, float balance_coef,
                                             float z_coef, float* losses) {
  losses[0] = all > 0 ? (float)(balance_coef * v[0] / all) : 0.0f;
  losses[1] = all > 0 ? (float)(z_coef * v[1] / all) : 0.0f;
}

// The sweep over the logits: a block's sums go to `sums`, and the block that is
// the last to have written its own takes the losses from all.  What the
// blocks hand each other passes the caches that they do not share (accesses of
// agent scope), and a block's sums have arrived (vmcnt 0) before its ticket is
// drawn: a fence would write back a whole L2 for them, 30 us for 1024 blocks.
// A ticket costs 7 ns, so the blocks are few and large.  (16384 x 768: 13 us, 3.8
// TB/s, some of it from the last cache.)
template <int W, int N, int VEC>
__global__ __launch_bounds__(kLossThreads) void balance_rows(
    const float* __restrict__ logits, const int32_t* __restrict__ seq, int n_seq, int T, int E,
    const float* __restrict__ load, const int32_t* __restrict__ tokens, float balance_coef,
    float z_coef, double* sums, unsigned* ticket, float* __restrict__ losses) {
  constexpr int kRows = kLossThreads / W;
  __shared__ double part[2][kLossThreads / kWave];
  __shared__ bool last;
  double v[2];
  loss_rows<W, N, VEC>(logits, seq, n_seq, T, E, load,
                       (long long)blockIdx.x * kRows + threadIdx.x / W,
                       (long long)gridDim.x * kRows, v);
  join_losses(v, part);
  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k)
      __hip_atomic_store(&sums[2 * blockIdx.x + k], v[k], __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");
    wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
           gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  for (int k = 0; k < 2; ++k)
    v[k] = threadIdx.x < gridDim.x   // kLossBlocks of them at most
               ? __hip_atomic_load(&sums[2 * threadIdx.x + k], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT)
               : 0.0;
  join_losses(v, part);
  if (threadIdx.x == 0) write_losses(v, tokens[n_seq], balance_coef, z_coef, losses);
}

// All of it by one block, for one sequence of few rows.
template <int W, int N, int VEC>
__global__ __launch_bounds__(kLossThreads) void balance_alone(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const int32_t* __restrict__ seq, const int32_t* __restrict__ group, int T, int E, int K,
    float balance_coef, float z_coef, int32_t* counts, int32_t* tokens, float* load,
    float* __restrict__ losses) {
  static_assert(kLossThreads == kCountThreads, "one block counts and sums");
  __shared__ CountLds lds;
  __shared__ double part[2][kLossThreads / kWave];
  count_sequence(0, lds, idx, seq, 1, group, T, E, K, counts, tokens, load);
  __syncthreads();   // the loads that this block has written, to all of it
  double v[2];
  loss_rows<W, N, VEC>(logits, seq, 1, T, E, load, threadIdx.x / W, kLossThreads / W, v);
  join_losses(v, part);
  if (threadIdx.x == 0) write_losses(v, lds.all, balance_coef, z_coef, losses);
}

// d_logits may be logits: a group has read the row that it overwrites.
template <int W, int N, int VEC>
__global__ __launch_bounds__(kThreads) void route_backward(
    const float* logits, const int32_t* __restrict__ idx, const float* __restrict__ d_gate,
    const int32_t* __restrict__ seq, int n_seq, const int32_t* __restrict__ tokens,
    const float* __restrict__ load, const float* __restrict__ d_losses, float balance_coef,
    float z_coef, int T, int E, int K, float* d_logits) {
  typedef RowOf<W, N, VEC> Row;
  constexpr int kRows = kThreads / W;   // rows of a block at a time
  __shared__ __attribute__((aligned(16))) float gates[kThreads * N * VEC];
  const int l = threadIdx.x % W, row = threadIdx.x / W;
  float* mine = gates + row * Row::kSize;   // the gates' gradient by expert, zeros between rows
  if (d_gate) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) mine[Row::at(i, l) + j] = 0.0f;
  }
  float cb = 0.0f, cz = 0.0f;
  if (load) {
    const int all = tokens[n_seq];
    if (all > 0) {
      cb = balance_coef * (d_losses ? d_losses[0] : 1.0f) / (float)all;
      cz = 2.0f * z_coef * (d_losses ? d_losses[1] : 1.0f) / (float)all;
    }
  }
  for (long long t = (long long)blockIdx.x * kRows + row; t < T;
       t += (long long)gridDim.x * kRows) {
    float p[N][VEC], g[N][VEC], f[N][VEC];
    Row::load(logits + t * E, E, l, p, -INFINITY);
    const int s = load ? sequence(seq, n_seq, t) : -1;
    if (s >= 0) Row::load(load + (size_t)s * E, E, l, f, 0.0f);
    if (d_gate) {
      wave_lds_order();
      for (int k0 = 0; k0 < K; k0 += W) {
        const int k = k0 + l;
        int e = k < K ? idx[t * K + k] : -1;
        const float d = k < K ? d_gate[t * K + k] : 0.0f;
        if (e >= E) e = -1;
        // whether two picks of the row are one expert: its lanes' numbers meet
        bool alone = K <= W;
        if (alone) {
          if (e >= 0) mine[e] = __int_as_float(l);
          wave_lds_order();
          alone = __ballot(e >= 0 && __float_as_int(mine[e]) != l) == 0;
          wave_lds_order();
          if (e >= 0) mine[e] = alone ? d : 0.0f;
          wave_lds_order();
        }
        if (!alone)   // one after the other: equal picks add up in their order
          for (int j = 0; j < W; ++j) {
            if (l == j && e >= 0) mine[e] += d;
            wave_lds_order();
          }
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[i][j] = mine[Row::at(i, l) + j];
      wave_lds_order();
      for (int k = l; k < K; k += W) {
        const int e = idx[t * K + k];
        if (e >= 0 && e < E) mine[e] = 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) g[i][j] = 0.0f;
    }
    const float lse = Row::softmax(p);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (s >= 0) g[i][j] = fmaf(cb, f[i][j], g[i][j]);
        if (p[i][j] == 0.0f) g[i][j] = 0.0f;   // a masked expert's may be anything
        dot = fmaf(p[i][j], g[i][j], dot);
      }
    dot = group_sum<W>(dot);
    const float more = s >= 0 ? cz * lse : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)   // and so may the others' sum
        p[i][j] = p[i][j] == 0.0f ? 0.0f : p[i][j] * (g[i][j] - dot + more);
    Row::store(d_logits + t * E, E, l, p);
  }
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// The narrowest groups of lanes that hold a row, four values a lane and load
// where rows and pointers allow.  (Gradient of 4096 x 96: 4.2 us with 32 lanes a
// row and four values a load, 5.9 with 64 and one.)
#define MOE_ROW_SHAPE(E, vec4, CALL)            \
  do {                                          \
    if (vec4) {                                 \
      if ((E) <= 32) { CALL(8, 1, 4); }         \
      else if ((E) <= 64) { CALL(16, 1, 4); }   \
      else if ((E) <= 128) { CALL(32, 1, 4); }  \
      else if ((E) <= 256) { CALL(64, 1, 4); }  \
      else if ((E) <= 512) { CALL(64, 2, 4); }  \
      else if ((E) <= 768) { CALL(64, 3, 4); }  \
      else { CALL(64, 4, 4); }                  \
    } else {                                    \
      if ((E) <= 8) { CALL(8, 1, 1); }          \
      else if ((E) <= 16) { CALL(16, 1, 1); }   \
      else if ((E) <= 32) { CALL(32, 1, 1); }   \
      else if ((E) <= 64) { CALL(64, 1, 1); }   \
      else if ((E) <= 128) { CALL(64, 2, 1); }  \
      else if ((E) <= 256) { CALL(64, 4, 1); }  \
      else if ((E) <= 512) { CALL(64, 8, 1); }  \
      else if ((E) <= 768) { CALL(64, 12, 1); } \
      else { CALL(64, 16, 1); }                 \
    }                                           \
  } while (0)

constexpr size_t kTicketBytes = 256;
constexpr long long kSequencePicks = 32768, kSequenceTokens = 1 << 22;

}  // namespace

size_t balance_ws_bytes() {
  return kTicketBytes + kLossBlocks * 2 * sizeof(double);
}

hipError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* seq,
                               int n_seq, const int32_t* group, int T, int E, int K,
                               float balance_coef, float z_coef, int32_t* counts, int32_t* tokens,
                               float* load, float* losses, void* ws, hipStream_t s) {
  unsigned* ticket = (unsigned*)ws;
  double* sums = (double*)((char*)ws + kTicketBytes);
  // One launch for one sequence of so few rows that a block takes them in four
  // turns (24, 96 and 768 experts: 7.9, 8.0 and 9.8 us at four, 9.3, 10.2 and 15.1 at
  // eight; in two launches 10.8 at either).
#define MOE_ALONE(W, N, VEC)                                                                   \
  if (n_seq == 1 && (long long)T * W <= 4 * kLossThreads) {                                    \
    MOE_LAUNCH("balance_alone", s,                                                             \
               balance_alone<W, N, VEC><<<1, kLossThreads, 0, s>>>(                            \
                   logits, idx, seq, group, T, E, K, balance_coef, z_coef, counts, tokens,     \
                   load, losses));                                                             \
    return hipGetLastError();                                                                  \
  }
  const bool vec4 = E % 4 == 0 && aligned16(logits) && aligned16(load);
  MOE_ROW_SHAPE(E, vec4, MOE_ALONE);
#undef MOE_ALONE
  // One launch where a block may count all picks and look at all tokens of every
  // sequence.  The losses in us, so and with three launches: 32768 picks 16.0 and 17.1
  // of one sequence, 11.6 and 17.4 of 16; 49152 picks 20.7 and 16.8, 15.1 and 17.2.
  // 32768 picks, 2^22 looks 15.3 and 18.9 (K 8) and 15.9 and 31.1 (K 2), 2^24 32.3 and
  // 20.5, 22.9 and 20.7.
  if ((long long)T * K <= kSequencePicks && (long long)T * n_seq <= kSequenceTokens) {
    MOE_LAUNCH("balance_count", s,
               balance_count_sequence<<<n_seq, kCountThreads, 0, s>>>(
                   idx, seq, n_seq, group, T, E, K, counts, tokens, load, ticket));
  } else {
    const long long n = std::max((long long)n_seq * E, (long long)n_seq + 1);
    MOE_LAUNCH("balance_clear", s,
               balance_clear<<<ceil_div(n, kThreads), kThreads, 0, s>>>(
                   counts, (long long)n_seq * E, tokens, n_seq + 1, ticket));
    MOE_LAUNCH("balance_count", s,
               balance_count<<<std::min(ceil_div(T, kCountTokens), kCountBlocks), kCountThreads, 0, s>>>(
                   idx, seq, n_seq, T, E, K, counts, tokens));
    MOE_LAUNCH("balance_load", s,
               balance_load<<<n_seq, kCountThreads, 0, s>>>(counts, tokens, group, E, K, load));
  }
#define MOE_BALANCE(W, N, VEC)                                                                 \
  MOE_LAUNCH("balance_rows", s,                                                                \
             balance_rows<W, N, VEC>                                                           \
                 <<<std::min(ceil_div(T, kLossThreads / W), kLossBlocks), kLossThreads, 0, s>>>( \
                     logits, seq, n_seq, T, E, load, tokens, balance_coef, z_coef, sums,       \
                     ticket, losses))
  MOE_ROW_SHAPE(E, vec4, MOE_BALANCE);
#undef MOE_BALANCE
  return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, const int32_t* idx, const float* d_gate,
                                 const int32_t* seq, int n_seq, const int32_t* tokens,
                                 const float* load, const float* d_losses, float balance_coef,
                                 float z_coef, int T, int E, int K, float* d_logits,
                                 hipStream_t s) {
#define MOE_BACKWARD(W, N, VEC)                                                                \
  MOE_LAUNCH("route_backward", s,                                                              \
             route_backward<W, N, VEC>                                                         \
                 <<<std::min(ceil_div(T, kThreads / W), kGradientBlocks), kThreads, 0, s>>>(   \
                     logits, idx, d_gate, seq, n_seq, tokens, load, d_losses, balance_coef,    \
                     z_coef, T, E, K, d_logits))
  MOE_ROW_SHAPE(E, E % 4 == 0 && aligned16(logits) && aligned16(load) && aligned16(d_logits),
                MOE_BACKWARD);
#undef MOE_BACKWARD
  return hipGetLastError();
}

}  // namespace moe

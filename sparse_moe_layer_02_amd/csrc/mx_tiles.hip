// The work list of the grouped 4-bit products, and which kernel takes what.
#include <algorithm>

#include "block_internal.h"
#include "mx_gemm.h"

namespace moe {
namespace mx {
namespace {

constexpr int kListThreads = 1024;
constexpr size_t kHeader = 256;

inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
// m-tiles of bm rows at most; workspaces hold the list of either form of rows
inline int tile_rows(bool fp4_rows) { return fp4_rows ? kMaxRows<true> : kMaxRows<false>; }
inline size_t max_tiles(int rows_cap, int n_experts, int bm) {
  return (size_t)rows_cap / bm + n_experts;
}

// The m-tiles of all experts, those of more than 64 rows first, then those of
// 17 to 64, then the rest; head[0..3]: where each part starts and the last
// ends.  An expert of m rows has m / bm full m-tiles and a rest.  Rows are
// clamped to [0, rows_cap) and the list to its capacity, so malformed offsets
// shrink the work but never index past the buffers.
__global__ __launch_bounds__(kListThreads) void mx_tiles(const int32_t* __restrict__ offsets,
                                                         int n_experts, int rows_cap, int bm,
                                                         int max_tiles, int* __restrict__ head,
                                                         int4* __restrict__ tiles) {
  constexpr int kParts = 3;
  __shared__ int wave_sum[kParts][kListThreads / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int per = (n_experts + kListThreads - 1) / kListThreads;
  const int lo = min(n_experts, tid * per), hi = min(n_experts, lo + per);
  auto span = [&](int e, int& r0, int& m) {
    r0 = min(max(offsets[e], 0), rows_cap);
    m = min(max(offsets[e + 1], r0), rows_cap) - r0;
  };
  auto part_of = [](int rows) { return rows > kMidRows ? 0 : rows > kSmallRows ? 1 : 2; };
  int mine[kParts] = {0, 0, 0}, sum[kParts];
  for (int e = lo; e < hi; ++e) {
    int r0, m;
    span(e, r0, m);
    const int rest = m % bm, k = part_of(rest);
    mine[0] += m / bm;
#pragma unroll
    for (int i = 0; i < kParts; ++i) mine[i] += rest > 0 && k == i ? 1 : 0;
  }
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    sum[i] = mine[i];                    // inclusive over the wave's lanes
    for (int off = 1; off < kWave; off <<= 1) {
      const int v = __shfl_up(sum[i], off);
      if (lane >= off) sum[i] += v;
    }
    if (lane == kWave - 1) wave_sum[i][wave] = sum[i];
  }
  __syncthreads();
  int at[kParts], end[kParts], start = 0;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    int before = 0, all = 0;
    for (int w = 0; w < kListThreads / kWave; ++w) {
      if (w == wave) before = all;
      all += wave_sum[i][w];
    }
    at[i] = start + before + sum[i] - mine[i];
    if (tid == 0) head[i] = start;
    start = end[i] = min(start + all, max_tiles);
  }
  if (tid == 0) head[kParts] = start;
  for (int e = lo; e < hi; ++e) {
    int r0, m;
    span(e, r0, m);
    for (int j = 0; j < m; j += bm) {
      const int rows = min(bm, m - j), k = part_of(rows);
#pragma unroll
      for (int i = 0; i < kParts; ++i)
        if (k == i) {
          if (at[i] < end[i]) tiles[at[i]] = make_int4(e, r0 + j, rows, 0);
          ++at[i];
        }
    }
  }
}

}  // namespace

size_t tile_list_bytes(int rows_cap, int n_experts) {
  return kHeader + align256(max_tiles(rows_cap, n_experts, kMaxRows<false>) * sizeof(int4));
}

bool grid_fits(int rows_cap, int n_experts, int N) {
  const long long m = (long long)max_tiles(rows_cap, n_experts, kMaxRows<false>) + 8;
  return m * (ceil_div((size_t)N, 64) + 1) < (1ll << 31) / kThreads;
}

hipError_t launch_tiles(const int32_t* offsets, int rows_cap, int n_experts, int rows_max,
                        bool fp4_rows, void* ws, hipStream_t s) {
  const int bm = tile_rows(fp4_rows);
  if (rows_max <= kSmallRows) return hipSuccess;   // one m-tile an expert, found by its number
  MOE_LAUNCH("mx_tiles", s,
             mx_tiles<<<1, kListThreads, 0, s>>>(offsets, n_experts, rows_cap, bm,
                                                 (int)max_tiles(rows_cap, n_experts, bm), (int*)ws,
                                                 (int4*)((char*)ws + kHeader)));
  return hipGetLastError();
}

hipError_t launch_product(const void* a, const uint8_t* a_scales, const int32_t* row_src, int T,
                          int K, const int32_t* offsets, int rows_cap, int n_experts, int rows_max,
                          int D, int N, const uint8_t* w, const uint8_t* w_scales, bool swiglu,
                          int out_dtype, void* out, void* ws, hipStream_t s) {
  GemmArgs p{};
  p.a = a;
  p.a_scales = a_scales;
  p.row_src = row_src;
  p.K = K;
  p.T = T;
  p.offsets = offsets;
  p.rows_cap = rows_cap;
  p.n_experts = n_experts;
  p.D = D;
  p.N = N;
  p.w = w;
  p.w_scales = w_scales;
  p.out = out;
  const bool fp4 = a_scales != nullptr;
  auto launch = [&](int kind, int cb, size_t mtiles) {
    return fp4 ? launch_gemm<true>(p, kind, swiglu, out_dtype, cb, (unsigned)mtiles, s)
               : launch_gemm<false>(p, kind, swiglu, out_dtype, cb, (unsigned)mtiles, s);
  };
  const size_t E = (size_t)n_experts, cap = (size_t)rows_cap;
  hipError_t e = hipSuccess;
  if (rows_max > kSmallRows) {
    const int* head = (const int*)ws;
    p.tiles = (const int4*)((char*)ws + kHeader);
    // grids by what the rows allow at most: a part's m-tiles hold so many rows
    // each, and an expert has one m-tile that is not full
    if (rows_max > kMidRows) {
      p.span = head;
      e = launch(2, 4, std::min(cap / (kMidRows + 1), cap / tile_rows(fp4) + E));
    }
    p.span = head + 1;
    if (e == hipSuccess) e = launch(1, 4, std::min(cap / (kSmallRows + 1), E));
    if (e != hipSuccess) return e;
    p.span = head + 2;
  }
  const size_t hit = std::min(cap, E);           // experts with rows, at most
  const size_t blocks4 = hit * ceil_div(N, 256);
  const int cb = blocks4 >= 512 ? 4 : 2 * blocks4 >= 512 || swiglu ? 2 : 1;
  return launch(0, cb, p.span ? hit : E);
}

}  // namespace mx
}  // namespace moe

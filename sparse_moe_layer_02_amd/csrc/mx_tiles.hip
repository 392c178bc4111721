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
// Whether the experts have few rows each, as far as the host can tell, which
// sees the buffer and not the rows in it: no expert more than 16, or at most 8
// rows of the buffer an expert and none over 128.  An expert that does have
// many is read past the caches once for every 16 rows.  Experts of 6144 x 2048,
// 45 of 64 with one row and one with m, in microseconds, this way against the
// list: m = 1: 166, 193; 16: 160, 193; 32: 179, 193; 64: 219, 207; 128: 327,
// 237.  The same batch (64 tokens, K 12, 64 of 768 experts) takes 162-170 in a
// buffer of 120 rows and 191-195 in one of 768, which is over 8 an expert.
inline bool few_rows(int rows_cap, int n_experts, int rows_max) {
  return rows_max <= kFewRows || (rows_max <= 128 && (long long)rows_cap <= 8ll * n_experts);
}
inline size_t max_tiles(int rows_cap, int n_experts, int bm) {
  return (size_t)rows_cap / bm + n_experts;
}

// The m-tiles of all experts, the largest first so that the small ones fill the
// end: those of more than 64 rows, of 17 to 64, and the rest; *count: how many.
// An expert of m rows has m / bm full m-tiles and a rest.  Rows are clamped to
// [0, rows_cap) and the list to its capacity, so malformed offsets shrink the
// work but never index past the buffers.
__global__ __launch_bounds__(kListThreads) void mx_tiles(const int32_t* __restrict__ offsets,
                                                         int n_experts, int rows_cap, int bm,
                                                         int max_tiles, int* __restrict__ count,
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
  auto part_of = [](int rows) { return rows > 64 ? 0 : rows > 16 ? 1 : 2; };
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
    start = end[i] = min(start + all, max_tiles);
  }
  if (tid == 0) *count = start;
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
  if (few_rows(rows_cap, n_experts, rows_max)) return hipSuccess;   // found by every block itself
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
  int few_cb = 0;
  size_t mtiles = max_tiles(rows_cap, n_experts, tile_rows(fp4));
  if (few_rows(rows_cap, n_experts, rows_max)) {
    mtiles = (size_t)std::min(rows_cap, n_experts);   // experts with rows, at most
    // 128 weight rows a block (two 16-row blocks a wave) where that gives every
    // CU its two, else 64.  256 rows a block were slower at every size (decode
    // FFN 189 against 167 us): fewer blocks to even out over the CUs.
    few_cb = swiglu || mtiles * ceil_div(N, 128) >= 512 ? 2 : 1;
  } else {
    p.tiles = (const int4*)((char*)ws + kHeader);
    p.count = (const int*)ws;
  }
  return fp4 ? launch_gemm<true>(p, few_cb, swiglu, out_dtype, (unsigned)mtiles, s)
             : launch_gemm<false>(p, few_cb, swiglu, out_dtype, (unsigned)mtiles, s);
}

}  // namespace mx
}  // namespace moe

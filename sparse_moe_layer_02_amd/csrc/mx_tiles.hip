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

// head: [0] m-tiles of more than 32 rows, [1] m-tiles of at most 32, [2] = 0
// (where the first start), [3] = head[0] (where the others start).
// An expert of m rows has m / bm full m-tiles and a rest.  Rows are clamped
// to [0, rows_cap) and the list to its capacity, so malformed offsets shrink
// the work but never index past the buffers.
__global__ __launch_bounds__(kListThreads) void mx_tiles(const int32_t* __restrict__ offsets,
                                                         int n_experts, int rows_cap, int bm,
                                                         int max_tiles, int* __restrict__ head,
                                                         int4* __restrict__ tiles) {
  __shared__ int2 wave_sum[kListThreads / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int per = (n_experts + kListThreads - 1) / kListThreads;
  const int lo = min(n_experts, tid * per), hi = min(n_experts, lo + per);
  auto span = [&](int e, int& r0, int& m) {
    r0 = min(max(offsets[e], 0), rows_cap);
    m = min(max(offsets[e + 1], r0), rows_cap) - r0;
  };
  int2 mine = make_int2(0, 0);
  for (int e = lo; e < hi; ++e) {
    int r0, m;
    span(e, r0, m);
    const int rest = m % bm;
    mine.x += m / bm + (rest > kSmallRows ? 1 : 0);
    mine.y += rest > 0 && rest <= kSmallRows ? 1 : 0;
  }
  int2 sum = mine;                       // inclusive over the wave's lanes
  for (int off = 1; off < kWave; off <<= 1) {
    const int x = __shfl_up(sum.x, off), y = __shfl_up(sum.y, off);
    if (lane >= off) {
      sum.x += x;
      sum.y += y;
    }
  }
  if (lane == kWave - 1) wave_sum[wave] = sum;
  __syncthreads();
  int2 before = make_int2(0, 0), all = make_int2(0, 0);
  for (int w = 0; w < kListThreads / kWave; ++w) {
    if (w == wave) before = all;
    all.x += wave_sum[w].x;
    all.y += wave_sum[w].y;
  }
  const int nl = min(all.x, max_tiles), ns = min(all.y, max_tiles - nl);
  int pl = before.x + sum.x - mine.x, ps = before.y + sum.y - mine.y;
  for (int e = lo; e < hi; ++e) {
    int r0, m;
    span(e, r0, m);
    const int mt = (m + bm - 1) / bm;
    for (int j = 0; j < mt; ++j) {
      const int rows = min(bm, m - j * bm);
      const int4 t = make_int4(e, r0 + j * bm, rows, mt);
      if (rows > kSmallRows) {
        if (pl < nl) tiles[pl] = t;
        ++pl;
      } else {
        if (ps < ns) tiles[nl + ps] = t;
        ++ps;
      }
    }
  }
  if (tid == 0) {
    head[0] = nl;
    head[1] = ns;
    head[2] = 0;
    head[3] = nl;
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
  int* head = (int*)ws;
  const bool list = rows_max > kSmallRows;
  hipError_t e = hipSuccess;
  if (list) {
    p.tiles = (const int4*)((char*)ws + kHeader);
    p.count = head;
    p.first = head + 2;
    const unsigned m = (unsigned)max_tiles(rows_cap, n_experts, tile_rows(a_scales != nullptr));
    e = a_scales ? launch_gemm_large<true>(p, swiglu, out_dtype, m, s)
                 : launch_gemm_large<false>(p, swiglu, out_dtype, m, s);
    if (e != hipSuccess) return e;
    p.count = head + 1;
    p.first = head + 3;
  }
  // at most one m-tile of at most 32 rows an expert
  const unsigned hit = (unsigned)std::min(rows_cap, n_experts);
  const unsigned blocks4 = hit * ceil_div(N, 256);
  const int cb = blocks4 >= 512 ? 4 : 2 * blocks4 >= 512 ? 2 : 1;
  return a_scales ? launch_gemm_small<true>(p, swiglu, out_dtype, cb, (unsigned)n_experts, s)
                  : launch_gemm_small<false>(p, swiglu, out_dtype, cb, (unsigned)n_experts, s);
}

}  // namespace mx
}  // namespace moe

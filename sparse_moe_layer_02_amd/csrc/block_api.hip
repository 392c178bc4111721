// C-ABI entry points of include/moe_mi355x_block.h: host-side validation (no
// HIP call before it passes), then the kernels are enqueued on the caller's
// stream.
#include <algorithm>

#include "block_internal.h"

using namespace moe;

namespace {

constexpr int kMaxExperts = 4096;
constexpr int kMaxNorm = 32768;
constexpr long long kMaxRowValues = 1ll << 39;   // a row's address is 32 bits of 128 values

inline bool dtype_ok(int d) { return d == MOE_F32 || d == MOE_BF16; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool fits_i32(long long v) { return v >= 0 && v < (1ll << 31); }
inline bool finite(float v) { return v == v && v - v == 0.0f; }
inline size_t al256(size_t b) { return (b + 255) & ~(size_t)255; }
inline moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// Sizes that the 4-bit rows of both conversions take.
inline bool rows_ok(long long rows, int cols) {
  return rows >= 1 && cols >= 1 && cols % 32 == 0 && rows < (1ll << 34) / cols;
}

// An expert's rows at most: with the dispatch indices one a token.
inline int rows_max(const int32_t* row_src, int rows_cap, int T) {
  return row_src ? std::min(rows_cap, T) : rows_cap;
}

moe_status product_sizes(const int32_t* row_src, int T, int K, int rows_cap, int n_experts, int D,
                         int N) {
  if (rows_cap < 1 || n_experts < 0 || n_experts > kMaxExperts || D < 1 || D % 128 || N < 1 ||
      N % 16 || !fits_i32((long long)N * D) || !mx::grid_fits(rows_cap, n_experts, N))
    return MOE_ERR_SHAPE;
  if (row_src && (T < 1 || K < 1 || !fits_i32((long long)T * K))) return MOE_ERR_SHAPE;
  if ((long long)(row_src ? T : rows_cap) * D > kMaxRowValues) return MOE_ERR_SHAPE;
  return MOE_OK;
}

struct FfnWs {
  void* list;
  void* hh;
  uint8_t* codes;
  uint8_t* scales;
  size_t total;
};

FfnWs ffn_ws(char* base, int rows_cap, int n_ffn, int I) {
  FfnWs w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += al256(bytes);
    return p;
  };
  w.list = take(mx::tile_list_bytes(rows_cap, n_ffn));
  w.hh = take((size_t)rows_cap * I * 2);
  w.codes = (uint8_t*)take((size_t)rows_cap * I / 2);
  w.scales = (uint8_t*)take((size_t)rows_cap * I / 32);
  w.total = off;
  return w;
}

}  // namespace

extern "C" {

moe_status moe_mxfp4_quantize(const void* x, int dtype, long long rows, int cols,
                              const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                              void* stream) {
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (!rows_ok(rows, cols)) return MOE_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(n_rows, 4))
    return MOE_ERR_ALIGN;
  return launched(launch_mxfp4_quantize(x, dtype, rows, cols, n_rows, codes, scales,
                                        (hipStream_t)stream));
}

moe_status moe_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                long long rows, int cols, void* y, void* stream) {
  if (!codes || !scales || !y) return MOE_ERR_NULL;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (!rows_ok(rows, cols)) return MOE_ERR_SHAPE;
  if (!aligned(y, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
  return launched(
      launch_mxfp4_dequantize(codes, scales, dtype, rows, cols, y, (hipStream_t)stream));
}

size_t moe_grouped_gemm_mxfp4_workspace_bytes(int rows_cap, int n_experts) {
  if (rows_cap < 1 || n_experts < 0 || n_experts > kMaxExperts) return 0;
  return mx::tile_list_bytes(rows_cap, n_experts);
}

moe_status moe_grouped_gemm_mxfp4(const void* a, const uint8_t* a_scales, const int32_t* row_src,
                                  int T, int K, const int32_t* offsets, int rows_cap,
                                  int n_experts, int D, int N, const uint8_t* w,
                                  const uint8_t* w_scales, int swiglu, int out_dtype, void* out,
                                  void* ws, size_t ws_bytes, void* stream) {
  if (!a || !offsets || !out || !ws || (n_experts != 0 && (!w || !w_scales))) return MOE_ERR_NULL;
  if (!dtype_ok(out_dtype)) return MOE_ERR_DTYPE;
  const moe_status st = product_sizes(row_src, T, K, rows_cap, n_experts, D, N);
  if (st != MOE_OK) return st;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(a_scales, 4) ||
      !aligned(w_scales, 4) || !aligned(offsets, 4) || !aligned(row_src, 4) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  if (ws_bytes < mx::tile_list_bytes(rows_cap, n_experts)) return MOE_ERR_WORKSPACE;
  if (n_experts == 0) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  const int most = rows_max(row_src, rows_cap, T);
  hipError_t e = mx::launch_tiles(offsets, rows_cap, n_experts, most, a_scales != nullptr, ws, s);
  if (e == hipSuccess)
    e = mx::launch_product(a, a_scales, row_src, T, K, offsets, rows_cap, n_experts, most, D, N, w,
                           w_scales, swiglu != 0, out_dtype, out, ws, s);
  return launched(e);
}

size_t moe_expert_ffn_mxfp4_workspace_bytes(int rows_cap, int n_ffn, int I) {
  if (rows_cap < 1 || n_ffn < 0 || n_ffn > kMaxExperts || I < 1) return 0;
  return ffn_ws(nullptr, rows_cap, n_ffn, I).total;
}

moe_status moe_expert_ffn_mxfp4(const void* x, const uint8_t* x_scales, int T, int K,
                                const int32_t* row_src, const int32_t* offsets, int rows_cap,
                                int n_ffn, int H, int I, const uint8_t* w13,
                                const uint8_t* w13_scales, const uint8_t* w2,
                                const uint8_t* w2_scales, void* y_perm, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!x || !row_src || !offsets || !y_perm || !ws ||
      (n_ffn != 0 && (!w13 || !w13_scales || !w2 || !w2_scales)))
    return MOE_ERR_NULL;
  if (I < 1 || I % 128 || !fits_i32(2ll * I)) return MOE_ERR_SHAPE;
  moe_status st = product_sizes(row_src, T, K, rows_cap, n_ffn, H, 2 * I);
  if (st == MOE_OK) st = product_sizes(nullptr, T, K, rows_cap, n_ffn, I, H);
  if (st != MOE_OK) return st;
  if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(y_perm, 16) ||
      !aligned(x_scales, 4) || !aligned(w13_scales, 4) || !aligned(w2_scales, 4) ||
      !aligned(row_src, 4) || !aligned(offsets, 4) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  const FfnWs f = ffn_ws((char*)ws, rows_cap, n_ffn, I);
  if (ws_bytes < f.total) return MOE_ERR_WORKSPACE;
  if (n_ffn == 0) return MOE_OK;
  const hipStream_t s = (hipStream_t)stream;
  const int most = rows_max(row_src, rows_cap, T);
  hipError_t e = mx::launch_tiles(offsets, rows_cap, n_ffn, most, x_scales != nullptr, f.list, s);
  // hh is rounded to bf16, as between the products of moe_expert_ffn: the matrix
  // cores multiply bf16 rows, and its remaining digits as rows of their own would
  // take twice the instructions in the down product.  It costs as much as the
  // output's own rounding: outputs are 0.0023 of their norm from the 64-bit form,
  // of which either rounding alone makes 0.0017.
  if (e == hipSuccess)
    e = mx::launch_product(x, x_scales, row_src, T, K, offsets, rows_cap, n_ffn, most, H, 2 * I,
                           w13, w13_scales, true, MOE_BF16, f.hh, f.list, s);
  if (e == hipSuccess && x_scales)
    e = launch_mxfp4_quantize(f.hh, MOE_BF16, rows_cap, I, offsets + n_ffn, f.codes, f.scales, s);
  if (e == hipSuccess)
    e = mx::launch_product(x_scales ? (const void*)f.codes : f.hh, x_scales ? f.scales : nullptr,
                           nullptr, 1, 1, offsets, rows_cap, n_ffn, most, I, H, w2, w2_scales,
                           false, MOE_BF16, y_perm, f.list, s);
  return launched(e);
}

moe_status moe_norm(const void* x, int x_dtype, const float* weight, float eps, int T, int H,
                    void* y, int y_dtype, void* stream) {
  if (!x || !y) return MOE_ERR_NULL;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return MOE_ERR_DTYPE;
  if (T < 1 || H < 1 || H % 8 || H > kMaxNorm || !finite(eps) || eps < 0.0f) return MOE_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16)) return MOE_ERR_ALIGN;
  return launched(launch_norm(x, x_dtype, weight, eps, T, H, y, y_dtype, (hipStream_t)stream));
}

moe_status moe_norm_residual(const void* y, int y_dtype, const float* w_post, float eps,
                             const float* gate, int gate_kind, float scale, const void* residual,
                             int res_dtype, void* res_out, const float* w_next, void* next, int T,
                             int H, void* stream) {
  if (!y || !residual || !res_out) return MOE_ERR_NULL;
  if (!dtype_ok(y_dtype) || !dtype_ok(res_dtype)) return MOE_ERR_DTYPE;
  if (T < 1 || H < 1 || H % 8 || H > kMaxNorm || !finite(eps) || eps < 0.0f || !finite(scale) ||
      gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_TOKEN)
    return MOE_ERR_SHAPE;
  if (gate_kind != MOE_GATE_NONE && !gate) return MOE_ERR_NULL;
  if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(res_out, 16) || !aligned(next, 16) ||
      !aligned(w_post, 16) || !aligned(w_next, 16) || !aligned(gate, 16))
    return MOE_ERR_ALIGN;
  return launched(launch_norm_residual(y, y_dtype, w_post, eps, gate, gate_kind, scale, residual,
                                       res_dtype, res_out, w_next, next, T, H,
                                       (hipStream_t)stream));
}

}  // extern "C"

// C-ABI entry points of include/moe_mi355x_train.h: host-side validation (no
// HIP call before it passes), then the kernels are enqueued on the caller's
// stream.
#include "train_internal.h"

using namespace moe;

namespace {

constexpr int kMaxNorm = 32768;
constexpr int kMaxSeq = 65536;

inline bool dtype_ok(int d) { return d == MOE_F32 || d == MOE_BF16; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool fits_i32(long long v) { return v >= 0 && v < (1ll << 31); }
inline bool finite(float v) { return v == v && v - v == 0.0f; }
inline moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

inline bool rows_ok(long long rows, int cols, int step) {
  return rows >= 1 && cols >= 1 && cols % step == 0 && rows <= ((1ll << 34) - 1) / cols;
}
inline bool norm_ok(int T, int H, float eps, bool mx8) {
  return T >= 1 && H >= 1 && H % (mx8 ? 32 : 8) == 0 && H <= kMaxNorm && finite(eps) &&
         eps >= 0.0f;
}
inline bool route_ok(int T, int E, const int32_t* seq, int n_seq, float balance_coef,
                     float z_coef) {
  return T >= 1 && E >= 1 && E <= kMaxRouteE && fits_i32((long long)T * E) && n_seq >= 1 &&
         n_seq <= kMaxSeq && (seq || n_seq == 1) && finite(balance_coef) && finite(z_coef);
}
inline bool picks_ok(int T, int E, int K) {
  return K >= 1 && K <= E && fits_i32((long long)T * K);
}

moe_status backward(bool mean, const void* dy, int dy_dtype, const void* x, int x_dtype,
                    const uint8_t* x_scales, const float* weight, float eps, int T, int H,
                    const void* d_residual, void* dx, int dx_dtype, float* d_weight, float* d_bias,
                    void* ws, size_t ws_bytes, void* stream) {
  const bool sums = d_weight || d_bias;
  if (!dy || !x || !dx || (sums && !ws)) return MOE_ERR_NULL;
  if (!dtype_ok(dy_dtype) || (!x_scales && !dtype_ok(x_dtype)) || !dtype_ok(dx_dtype))
    return MOE_ERR_DTYPE;
  if (!norm_ok(T, H, eps, x_scales != nullptr)) return MOE_ERR_SHAPE;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dx, 16) || !aligned(weight, 16) ||
      !aligned(d_residual, 16) || !aligned(d_weight, 16) || !aligned(d_bias, 16) ||
      !aligned(x_scales, 4) || !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  if (sums && ws_bytes < norm_backward_ws_bytes(T, H)) return MOE_ERR_WORKSPACE;
  return launched(launch_norm_backward(mean, dy, dy_dtype, x, x_dtype, x_scales, weight, eps, T, H,
                                       d_residual, dx, dx_dtype, d_weight, d_bias, ws,
                                       (hipStream_t)stream));
}

}  // namespace

extern "C" {

size_t moe_balance_loss_workspace_bytes(int T, int E, int n_seq) {
  if (T < 1 || E < 1 || E > kMaxRouteE || n_seq < 1 || n_seq > kMaxSeq) return 0;
  return balance_ws_bytes();
}

moe_status moe_balance_loss(const float* logits, const int32_t* topk_idx, const int32_t* seq,
                            int n_seq, const int32_t* group, int T, int E, int K,
                            float balance_coef, float z_coef, int32_t* counts, int32_t* tokens,
                            float* load, float* losses, void* ws, size_t ws_bytes, void* stream) {
  if (!logits || !topk_idx || !counts || !tokens || !load || !losses || !ws) return MOE_ERR_NULL;
  if (!route_ok(T, E, seq, n_seq, balance_coef, z_coef) || !picks_ok(T, E, K))
    return MOE_ERR_SHAPE;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(seq, 4) || !aligned(group, 4) ||
      !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(load, 4) || !aligned(losses, 4) ||
      !aligned(ws, 256))
    return MOE_ERR_ALIGN;
  if (ws_bytes < balance_ws_bytes()) return MOE_ERR_WORKSPACE;
  return launched(launch_balance_loss(logits, topk_idx, seq, n_seq, group, T, E, K, balance_coef,
                                      z_coef, counts, tokens, load, losses, ws,
                                      (hipStream_t)stream));
}

moe_status moe_route_backward(const float* logits, const int32_t* topk_idx, const float* d_gate,
                              const int32_t* seq, int n_seq, const int32_t* tokens,
                              const float* load, const float* d_losses, float balance_coef,
                              float z_coef, int T, int E, int K, float* d_logits, void* stream) {
  if (!logits || !d_logits || (!d_gate && !load) || (d_gate && !topk_idx) || (load && !tokens) ||
      (tokens && !load))
    return MOE_ERR_NULL;
  if (!route_ok(T, E, seq, n_seq, balance_coef, z_coef) || (d_gate && !picks_ok(T, E, K)))
    return MOE_ERR_SHAPE;
  if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(d_gate, 4) || !aligned(seq, 4) ||
      !aligned(tokens, 4) || !aligned(load, 4) || !aligned(d_losses, 4) || !aligned(d_logits, 4))
    return MOE_ERR_ALIGN;
  return launched(launch_route_backward(logits, topk_idx, d_gate, seq, n_seq, tokens, load,
                                        d_losses, balance_coef, z_coef, T, E, K, d_logits,
                                        (hipStream_t)stream));
}

moe_status moe_mxfp8_quantize(const void* x, int dtype, long long rows, int cols,
                              const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                              void* stream) {
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (!rows_ok(rows, cols, 32)) return MOE_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(n_rows, 4))
    return MOE_ERR_ALIGN;
  return launched(launch_mxfp8_quantize(x, dtype, rows, cols, n_rows, codes, scales,
                                        (hipStream_t)stream));
}

moe_status moe_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                long long rows, int cols, void* y, void* stream) {
  if (!codes || !scales || !y) return MOE_ERR_NULL;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (!rows_ok(rows, cols, 32)) return MOE_ERR_SHAPE;
  if (!aligned(y, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
  return launched(
      launch_mxfp8_dequantize(codes, scales, dtype, rows, cols, y, (hipStream_t)stream));
}

moe_status moe_norm_checkpoint(const void* x, int x_dtype, const float* weight, float eps, int T,
                               int H, void* y, int y_dtype, uint8_t* codes, uint8_t* scales,
                               void* stream) {
  if (!x || !y || !codes || !scales) return MOE_ERR_NULL;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return MOE_ERR_DTYPE;
  if (!norm_ok(T, H, eps, true)) return MOE_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return MOE_ERR_ALIGN;
  return launched(launch_norm_save(false, x, x_dtype, weight, nullptr, eps, T, H, y, y_dtype,
                                   codes, scales, (hipStream_t)stream));
}

moe_status moe_layer_norm(const void* x, int x_dtype, const float* weight, const float* bias,
                          float eps, int T, int H, void* y, int y_dtype, uint8_t* codes,
                          uint8_t* scales, void* stream) {
  if (!x || !y || (codes != nullptr) != (scales != nullptr)) return MOE_ERR_NULL;
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype)) return MOE_ERR_DTYPE;
  if (!norm_ok(T, H, eps, codes != nullptr)) return MOE_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(weight, 16) || !aligned(bias, 16) ||
      !aligned(codes, 16) || !aligned(scales, 4))
    return MOE_ERR_ALIGN;
  return launched(launch_norm_save(true, x, x_dtype, weight, bias, eps, T, H, y, y_dtype, codes,
                                   scales, (hipStream_t)stream));
}

size_t moe_norm_backward_workspace_bytes(int T, int H) {
  if (T < 1 || H < 1 || H > kMaxNorm) return 0;
  return norm_backward_ws_bytes(T, H);
}

moe_status moe_norm_backward(const void* dy, int dy_dtype, const void* x, int x_dtype,
                             const uint8_t* x_scales, const float* weight, float eps, int T, int H,
                             const void* d_residual, void* dx, int dx_dtype, float* d_weight,
                             void* ws, size_t ws_bytes, void* stream) {
  return backward(false, dy, dy_dtype, x, x_dtype, x_scales, weight, eps, T, H, d_residual, dx,
                  dx_dtype, d_weight, nullptr, ws, ws_bytes, stream);
}

moe_status moe_layer_norm_backward(const void* dy, int dy_dtype, const void* x, int x_dtype,
                                   const uint8_t* x_scales, const float* weight, float eps, int T,
                                   int H, const void* d_residual, void* dx, int dx_dtype,
                                   float* d_weight, float* d_bias, void* ws, size_t ws_bytes,
                                   void* stream) {
  return backward(true, dy, dy_dtype, x, x_dtype, x_scales, weight, eps, T, H, d_residual, dx,
                  dx_dtype, d_weight, d_bias, ws, ws_bytes, stream);
}

moe_status moe_swiglu(const void* gu, int dtype, long long rows, int I, const int32_t* n_rows,
                      void* hh, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!gu || !hh || (codes != nullptr) != (scales != nullptr)) return MOE_ERR_NULL;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (I < 1 || !fits_i32(2ll * I) || !rows_ok(rows, 2 * I, codes ? 64 : 16)) return MOE_ERR_SHAPE;
  if (!aligned(gu, 16) || !aligned(hh, 16) || !aligned(codes, 16) || !aligned(scales, 4) ||
      !aligned(n_rows, 4))
    return MOE_ERR_ALIGN;
  return launched(
      launch_swiglu(gu, dtype, rows, I, n_rows, hh, codes, scales, (hipStream_t)stream));
}

moe_status moe_swiglu_backward(const void* d_hh, const void* gu, const uint8_t* gu_scales,
                               int dtype, long long rows, int I, const int32_t* n_rows,
                               void* d_gu, void* hh, void* stream) {
  if (!d_hh || !gu || !d_gu) return MOE_ERR_NULL;
  if (!dtype_ok(dtype)) return MOE_ERR_DTYPE;
  if (I < 1 || !fits_i32(2ll * I) || !rows_ok(rows, 2 * I, gu_scales ? 64 : 16))
    return MOE_ERR_SHAPE;
  if (!aligned(d_hh, 16) || !aligned(gu, 16) || !aligned(d_gu, 16) || !aligned(hh, 16) ||
      !aligned(gu_scales, 4) || !aligned(n_rows, 4))
    return MOE_ERR_ALIGN;
  return launched(launch_swiglu_backward(d_hh, gu, gu_scales, dtype, rows, I, n_rows, d_gu, hh,
                                         (hipStream_t)stream));
}

}  // extern "C"

// Launchers of the routing losses, the norms' backward passes and the 8-bit
// activations (each returns hipGetLastError() after enqueueing).
#pragma once

#include "../../include/moe_mi355x_train.h"
#include "moe_internal.h"

namespace moe {

constexpr int kMaxRouteE = 1024;   // a wave's row: up to 16 logits a lane

size_t balance_ws_bytes();
hipError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* seq,
                               int n_seq, const int32_t* group, int T, int E, int K,
                               float balance_coef, float z_coef, int32_t* counts, int32_t* tokens,
                               float* load, float* losses, void* ws, hipStream_t s);
hipError_t launch_route_backward(const float* logits, const int32_t* idx, const float* d_gate,
                                 const int32_t* seq, int n_seq, const int32_t* tokens,
                                 const float* load, const float* d_losses, float balance_coef,
                                 float z_coef, int T, int E, int K, float* d_logits,
                                 hipStream_t s);

hipError_t launch_mxfp8_quantize(const void* x, int dtype, long long rows, int cols,
                                 const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s);
hipError_t launch_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                   long long rows, int cols, void* y, hipStream_t s);
hipError_t launch_swiglu(const void* gu, int dtype, long long rows, int I, const int32_t* n_rows,
                         void* hh, uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_swiglu_backward(const void* d_hh, const void* gu, const uint8_t* gu_scales,
                                  int dtype, long long rows, int I, const int32_t* n_rows,
                                  void* d_gu, void* hh, hipStream_t s);

// mean: by mean and variance (moe_layer_norm), else by root mean square.
hipError_t launch_norm_save(bool mean, const void* x, int x_dtype, const float* weight,
                            const float* bias, float eps, int T, int H, void* y, int y_dtype,
                            uint8_t* codes, uint8_t* scales, hipStream_t s);
size_t norm_backward_ws_bytes(int T, int H);
hipError_t launch_norm_backward(bool mean, const void* dy, int dy_dtype, const void* x,
                                int x_dtype, const uint8_t* x_scales, const float* weight,
                                float eps, int T, int H, const void* d_residual, void* dx,
                                int dx_dtype, float* d_weight, float* d_bias, void* ws,
                                hipStream_t s);

}  // namespace moe

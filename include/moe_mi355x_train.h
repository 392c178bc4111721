/*
 * moe_mi355x_train.h -- C ABI of what training adds around the MoE layer of
 * moe_mi355x.h and the norms of moe_mi355x_block.h: the losses that keep the
 * router balanced and the gradient of its logits, the norm by mean and
 * variance, the backward passes of the norms, and activations kept in 8 bits
 * from the forward to the backward pass.
 *
 * The conventions are those of moe_mi355x.h: device pointers owned by the
 * caller, kernels enqueued on `stream` without synchronising, arguments
 * checked on the host before any HIP call, status codes, row-major contiguous
 * tensors, bitwise the same results from run to run, no state between calls,
 * and calls that share a workspace ordered on one stream.  Outputs are
 * overwritten, never added to.
 *
 * MXFP8 (OCP Microscaling Formats (MX) v1.0, e4m3).  A row of C values,
 * C % 32 == 0, is held as C code bytes and C / 32 scale bytes, one for each
 * block of 32 values.  A code is a sign bit, 4 bits of exponent (bias 7) and 3
 * of mantissa, up to 448, without infinities (0x7f and 0xff are NaN); a scale
 * byte b is 2^(b - 127), and 255 makes all of its block NaN.
 */
#ifndef MOE_MI355X_TRAIN_H
#define MOE_MI355X_TRAIN_H

#include "moe_mi355x_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The losses of a batch's routing, and what its experts were given.
 *   p[t][e] = softmax of logits[t], lse[t] = log of the sum of their exp
 *   counts[s][e] = picks of expert e by the tokens of sequence s
 *   tokens[s]    = tokens of sequence s; tokens[n_seq] = those of all, N
 *   load[s][e]   = E * counts[s][e] / (K * tokens[s]), averaged over the
 *                  experts of e's group (1 where the picks are spread evenly;
 *                  0 in a sequence without tokens)
 *   losses[0] = balance_coef / N * sum over t, e of load[seq[t]][e] * p[t][e]
 *   losses[1] = z_coef / N * sum over t of lse[t]^2
 * logits [T][E] fp32; topk_idx [T][K] (ids outside [0, E) are no picks, equal
 * ids of a token count each); seq [T]: the token's sequence, any order, where an
 * id outside [0, n_seq) marks padding, which counts nowhere; NULL with n_seq
 * == 1: all tokens are sequence 0.  group [E]: the expert's group, an id in
 * [0, E), outside of which the expert is left out (load 0); NULL: every expert
 * by itself.  counts [n_seq][E], tokens [n_seq + 1], load [n_seq][E] fp32,
 * losses [2] fp32.
 * A logit of -inf is a masked expert; a token all of whose logits are -inf has
 * p = 0 and lse = 0 (but is a token).  A NaN or +inf in a counted token's
 * logits makes the losses NaN.  N == 0: both losses 0.
 * fp32 softmax, the sums over tokens in fp64.
 * MOE_ERR_SHAPE: T < 1, K outside 1..E, E > 1024, T*E or T*K >= 2^31, n_seq
 * outside 1..65536 or not 1 without seq, a coefficient that is not finite.
 * MOE_ERR_ALIGN: pointers 4 bytes, ws 256.
 * ws: at least moe_balance_loss_workspace_bytes(T, E, n_seq). */
size_t moe_balance_loss_workspace_bytes(int T, int E, int n_seq);
moe_status moe_balance_loss(const float *logits, const int32_t *topk_idx, const int32_t *seq,
                            int n_seq, const int32_t *group, int T, int E, int K,
                            float balance_coef, float z_coef, int32_t *counts, int32_t *tokens,
                            float *load, float *losses, void *ws, size_t ws_bytes, void *stream);

/* The gradient of moe_route's gates and of moe_balance_loss's losses with
 * respect to the logits (the picks, and so load, are constants of it):
 *   g[t][e] = sum over k with topk_idx[t][k] == e of d_gate[t][k]
 *           + balance_coef / N * d_losses[0] * load[seq[t]][e]
 *   d_logits[t][e] = p[t][e] * (g[t][e] - sum over j of p[t][j] * g[t][j]
 *           + 2 * z_coef / N * d_losses[1] * lse[t])
 * d_gate [T][K]: the gradient of topk_gate; NULL: gates have none (topk_idx
 * may then be NULL).  load, tokens: as moe_balance_loss wrote them; both NULL:
 * no losses.  One of d_gate and load has to be there.  seq, n_seq and the
 * coefficients: as for moe_balance_loss; padding has a gradient from its
 * d_gate alone.  d_losses [2] fp32 in device memory: the gradients of the two
 * losses; NULL: ones.  d_logits [T][E] fp32; it may be logits.
 * A masked expert's gradient is 0, whatever d_gate and d_losses hold (its
 * probability is 0), and so are those of a token whose logits are all -inf; a NaN
 * or +inf in a token's logits makes all of its row NaN.
 * Errors as for moe_balance_loss; K is only looked at with d_gate. */
moe_status moe_route_backward(const float *logits, const int32_t *topk_idx, const float *d_gate,
                              const int32_t *seq, int n_seq, const int32_t *tokens,
                              const float *load, const float *d_losses, float balance_coef,
                              float z_coef, int T, int E, int K, float *d_logits, void *stream);

/* Rows to MXFP8.  For each block of 32 values x_i with m = max |x_i|:
 *   scale  = the smallest power of two with m / scale <= 448, at least 2^-127
 *   code_i = x_i / scale rounded to e4m3, ties to the even code
 * so no value is clipped.  In a block whose scale is above 2^-127 the largest is
 * more than 224 scales, and a value within a factor of 7 * 2^11 of it, so of 2^-6
 * scales or more (e4m3's normal numbers), is off by at most 2^-4 of itself.  A
 * block that holds a NaN or an infinity gets scale byte 255 and NaN codes.
 *   x [rows][cols] (dtype, 16-byte aligned), codes [rows][cols] (16-byte
 *   aligned), scales [rows][cols / 32] (4-byte aligned).
 * n_rows: NULL, or one int32 in device memory: only the first
 * min(max(*n_rows, 0), rows) rows are converted and the others left as they
 * were.
 * MOE_ERR_SHAPE: rows < 1, cols < 1, cols % 32 != 0 or rows * cols >= 2^34. */
moe_status moe_mxfp8_quantize(const void *x, int dtype, long long rows, int cols,
                              const int32_t *n_rows, uint8_t *codes, uint8_t *scales,
                              void *stream);

/* The values that MXFP8 rows stand for, in dtype: exact in fp32; in bf16 too,
 * but for magnitudes below 2^-126, which are rounded (only blocks at the lowest
 * scales hold such values).  Magnitudes of 2^128 and more become infinities:
 * moe_mxfp8_quantize rounds finite ones from 1.9375 * 2^127 on to 2^128 (256 at
 * scale 2^120), and passes that read a checkpoint have infinities in their place.
 * y [rows][cols] (16-byte aligned); the rest as for moe_mxfp8_quantize. */
moe_status moe_mxfp8_dequantize(const uint8_t *codes, const uint8_t *scales, int dtype,
                                long long rows, int cols, void *y, void *stream);

/* moe_norm that leaves its input behind in 8 bits for the backward pass: y is
 * bitwise that of moe_norm, codes [T][H] and scales [T][H / 32] bitwise those
 * of moe_mxfp8_quantize on x.  y may be x when the dtypes are equal.
 * Errors as for moe_norm, MOE_ERR_SHAPE also for H % 32; codes 16-byte, scales
 * 4-byte aligned. */
moe_status moe_norm_checkpoint(const void *x, int x_dtype, const float *weight, float eps, int T,
                               int H, void *y, int y_dtype, uint8_t *codes, uint8_t *scales,
                               void *stream);

/* The norm by mean and variance:
 *   m[t] = mean over h of x[t][h],  v[t] = mean over h of (x[t][h] - m[t])^2
 *   y[t][h] = (x[t][h] - m[t]) / sqrt(v[t] + eps) * weight[h] + bias[h]
 * weight [H] fp32 or NULL (ones), bias [H] fp32 or NULL (zeros); codes and
 * scales: NULL, or x in 8 bits is left there as by moe_norm_checkpoint.  fp32
 * arithmetic, the deviations from the mean squared themselves and their own mean
 * taken out of them again, so that a row far from zero keeps the digits that its
 * values have of its spread; rows whose sums or squares fp32 cannot hold are
 * scaled by a power of two first.  A constant row gives the bias with eps > 0,
 * NaN with eps == 0.  y may be x when the dtypes are equal.
 * Errors as for moe_norm; with codes H % 32 == 0, and scales with codes. */
moe_status moe_layer_norm(const void *x, int x_dtype, const float *weight, const float *bias,
                          float eps, int T, int H, void *y, int y_dtype, uint8_t *codes,
                          uint8_t *scales, void *stream);

/* The backward pass of moe_norm.  With n = x * r, r = 1 / sqrt(mean(x^2) + eps)
 * of the row and g = dy * weight:
 *   dx = r * (g - n * mean over h of (g * n)) + d_residual
 *   d_weight[h] = sum over t of dy[t][h] * n[t][h]
 * dy [T][H] in dy_dtype.  x, in one of two forms: x_scales NULL: [T][H] in
 * x_dtype; else MXFP8, codes [T][H] and x_scales [T][H / 32] (x_dtype is not
 * looked at), and x is the values that they stand for.  The rows' roots are
 * taken again from x.  weight [H] fp32 or NULL (ones).  d_residual [T][H] in
 * dx_dtype: the gradient that reaches x beside the norm (the residual
 * stream's), or NULL.  dx [T][H] in dx_dtype; it may be d_residual, or x or dy
 * of the same dtype.  d_weight [H] fp32, or NULL where the weight has no
 * gradient (ws may then be NULL).
 * fp32 arithmetic; d_weight is a sum over rows in a fixed order that depends
 * on the sizes, the types and whether there is a d_residual.
 * MOE_ERR_SHAPE: T < 1, H < 1, H % 8 (MXFP8: H % 32), H > 32768, or eps
 * negative or not finite.  MOE_ERR_ALIGN: 16 bytes, x_scales 4, ws 256.
 * ws: at least moe_norm_backward_workspace_bytes(T, H). */
size_t moe_norm_backward_workspace_bytes(int T, int H);
moe_status moe_norm_backward(const void *dy, int dy_dtype, const void *x, int x_dtype,
                             const uint8_t *x_scales, const float *weight, float eps, int T, int H,
                             const void *d_residual, void *dx, int dx_dtype, float *d_weight,
                             void *ws, size_t ws_bytes, void *stream);

/* The backward pass of moe_layer_norm.  With n = (x - m) * r:
 *   dx = r * (g - mean(g) - n * mean(g * n)) + d_residual
 *   d_weight[h] = sum over t of dy[t][h] * n[t][h],  d_bias[h] = sum of dy[t][h]
 * d_bias [H] fp32 or NULL; the rest as for moe_norm_backward. */
moe_status moe_layer_norm_backward(const void *dy, int dy_dtype, const void *x, int x_dtype,
                                   const uint8_t *x_scales, const float *weight, float eps, int T,
                                   int H, const void *d_residual, void *dx, int dx_dtype,
                                   float *d_weight, float *d_bias, void *ws, size_t ws_bytes,
                                   void *stream);

/* The SwiGLU between an expert's two products, as a call of its own that keeps
 * its input in 8 bits for the backward pass:
 *   hh[r][j] = silu(gu[r][j]) * gu[r][I + j],  silu(a) = a / (1 + exp(-a))
 * gu [rows][2I] (dtype), hh [rows][I] (dtype); codes [rows][2I] and scales
 * [rows][2I / 32]: NULL, or gu in 8 bits as by moe_mxfp8_quantize.
 * n_rows as for moe_mxfp8_quantize (offsets + n_ffn takes the grouped rows).
 * fp32 arithmetic, rounded once; where exp(-a) passes 2^128 (a below -88.7, silu
 * above -3e-37) the output is 0.
 * MOE_ERR_SHAPE: rows < 1, I < 1, I % 8 (with codes I % 32) or rows * 2I >=
 * 2^34.  MOE_ERR_ALIGN: 16 bytes, scales and n_rows 4. */
moe_status moe_swiglu(const void *gu, int dtype, long long rows, int I, const int32_t *n_rows,
                      void *hh, uint8_t *codes, uint8_t *scales, void *stream);

/* The backward pass of moe_swiglu.  With s = 1 / (1 + exp(-g)):
 *   d_gu[r][j]     = d_hh[r][j] * u * s * (1 + g * (1 - s))
 *   d_gu[r][I + j] = d_hh[r][j] * g * s        g = gu[r][j], u = gu[r][I + j]
 * d_hh [rows][I] (dtype).  gu, in one of two forms: gu_scales NULL: [rows][2I]
 * (dtype); else MXFP8 codes [rows][2I] and gu_scales [rows][2I / 32].  d_gu
 * [rows][2I] (dtype); it may be gu of dtype.  hh: NULL, or [rows][I] (dtype):
 * moe_swiglu's output is computed again from gu (the rows of the down
 * product's weight gradient); it may be d_hh.
 * The rest as for moe_swiglu. */
moe_status moe_swiglu_backward(const void *d_hh, const void *gu, const uint8_t *gu_scales,
                               int dtype, long long rows, int I, const int32_t *n_rows,
                               void *d_gu, void *hh, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_TRAIN_H */

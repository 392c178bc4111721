/*
 * moe_mi355x_block.h -- C ABI of what surrounds the MoE layer of
 * moe_mi355x.h in a served block: its expert weights in microscaled 4-bit
 * floating point (MXFP4), and the norms before and after the block.
 *
 * The conventions are those of moe_mi355x.h: device pointers owned by the
 * caller, kernels enqueued on `stream` without synchronising, arguments
 * checked on the host before any HIP call, status codes, row-major contiguous
 * tensors, bitwise the same results from run to run, no state between calls,
 * and calls that share a workspace ordered on one stream.
 *
 * MXFP4 (OCP Microscaling Formats (MX) v1.0).  A row of C values, C % 32 ==
 * 0, is held as C / 2 bytes of codes (value 2i in the low half of byte i,
 * value 2i + 1 in the high half) and C / 32 scale bytes, one for each block
 * of 32 values.  A code is a sign bit (8) and an e2m1 magnitude 0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 (codes 0..7); a scale byte b is 2^(b - 127), and 255 makes
 * all of its block NaN.
 */
#ifndef MOE_MI355X_BLOCK_H
#define MOE_MI355X_BLOCK_H

#include "moe_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows to MXFP4.  For each block of 32 values x_i with m = max |x_i|:
 *   scale = 2^(floor(log2 m) - 2), at least 2^-127 (m = 0: 2^-127),
 *   code_i = x_i / scale rounded to e2m1, ties to the even code, magnitudes
 *            over 6 to 6 (m / scale lies in [4, 8)).
 * A block that holds a NaN or an infinity gets scale byte 255 and codes that
 * mean nothing.
 *   x [rows][cols] (dtype, 16-byte aligned), codes [rows][cols / 2] (16-byte
 *   aligned), scales [rows][cols / 32] (4-byte aligned).
 * n_rows: NULL, or one int32 in device memory: only the first
 * min(max(*n_rows, 0), rows) rows are converted and the others left as they
 * were (offsets + n_ffn converts the rows that moe_permute grouped).
 * MOE_ERR_SHAPE: rows < 1, cols < 1, cols % 32 != 0 or rows * cols >= 2^34. */
moe_status moe_mxfp4_quantize(const void *x, int dtype, long long rows, int cols,
                              const int32_t *n_rows, uint8_t *codes, uint8_t *scales,
                              void *stream);

/* The values that MXFP4 rows stand for, in dtype: exact in fp32 and in bf16,
 * but for magnitudes of 2^128 and more, which become infinities (4 and 6 at
 * scale byte 253, 2 to 6 at 254; moe_mxfp4_quantize writes no scale byte over
 * 252 but 255).
 * y [rows][cols] (16-byte aligned); the rest as for moe_mxfp4_quantize. */
moe_status moe_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int dtype,
                                long long rows, int cols, void *y, void *stream);

/* Matrix products grouped by expert on MXFP4 weights.  For every expert e and
 * row r in [offsets[e], offsets[e + 1]) (empty experts cost nothing):
 *   c[n] = sum over d of a(r)[d] * w[e][n][d],  n < N, fp32 accumulation
 *   out[r] = c, or with swiglu silu(c[j]) * c[N / 2 + j] for j < N / 2
 * a: the rows, in one of two forms:
 *   a_scales NULL: bf16 [.][D].  The weights count as bf16 values too, those
 *     of 2^128 and more as infinities (as in moe_mxfp4_dequantize);
 *   else MXFP4: codes [.][D / 2] in a, scales [.][D / 32] in a_scales.  Every
 *     product is that of the values themselves.
 * row_src: NULL, and a(r) = a[r] with rows_cap rows in a; or the dispatch
 *   indices of moe_permute (capacity rows_cap), and a(r) = a[row_src[r] / K]
 *   with T rows in a (indices outside [0, T*K) are clamped to a row of a).
 *   K and T are only looked at with row_src.
 * offsets [n_experts + 1] int32 with offsets[n_experts] <= rows_cap (spans are
 *   clamped into [0, rows_cap]); a row past the last span is left as it was.
 * w [n_experts][N][D / 2] codes, w_scales [n_experts][N][D / 32].
 * out [rows_cap][N] (swiglu: [rows_cap][N / 2]) in out_dtype.
 * MOE_ERR_SHAPE: rows_cap < 1, n_experts outside 0..4096, D < 1 or D % 128,
 *   N < 1 or N % 16, N * D >= 2^31, T < 1, K < 1 or T*K >= 2^31 with row_src,
 *   more than 2^39 values in the rows of a (T * D with row_src, rows_cap * D
 *   without), or more blocks than a launch takes.
 * MOE_ERR_ALIGN: a, w, out 16 bytes; a_scales, w_scales, offsets, row_src 4;
 *   ws 256.  n_experts == 0 enqueues nothing (w, w_scales may be NULL).
 * ws: at least moe_grouped_gemm_mxfp4_workspace_bytes(rows_cap, n_experts).
 * The kernel is chosen by the sizes alone: the one for small batches with at
 * most 16 rows an expert (rows_cap, or with row_src T, at most 16), or with at
 * most 128 and rows_cap <= 8 * n_experts.  A batch of few rows runs faster in a
 * buffer within that. */
size_t moe_grouped_gemm_mxfp4_workspace_bytes(int rows_cap, int n_experts);
moe_status moe_grouped_gemm_mxfp4(const void *a, const uint8_t *a_scales, const int32_t *row_src,
                                  int T, int K, const int32_t *offsets, int rows_cap,
                                  int n_experts, int D, int N, const uint8_t *w,
                                  const uint8_t *w_scales, int swiglu, int out_dtype, void *out,
                                  void *ws, size_t ws_bytes, void *stream);

/* moe_expert_ffn_gather on MXFP4 weights: two grouped products with the
 * SwiGLU between them,
 *   hh = silu(X W_g^T) * (X W_u^T),  y_perm rows = hh W_d^T,
 * w13 [n_ffn][2I][H / 2] codes and w13_scales [n_ffn][2I][H / 32], w2
 * [n_ffn][H][I / 2] and w2_scales [n_ffn][H][I / 32].
 * x_scales NULL: x is bf16 [T][H], and hh is rounded to bf16.  Else x and
 * x_scales are MXFP4 rows, and hh, rounded to bf16, is converted to MXFP4 as
 * by moe_mxfp4_quantize (y_perm is bitwise that of the three calls).
 * y_perm [rows_cap][H] bf16; rows past offsets[n_ffn] are left as they were.
 * T, K, row_src, offsets, rows_cap as for moe_expert_ffn_gather.
 * MOE_ERR_SHAPE also for H % 128 or I % 128, for 2 * I * H >= 2^31 and for
 * T * H or rows_cap * I past 2^39.
 * ws: at least moe_expert_ffn_mxfp4_workspace_bytes(rows_cap, n_ffn, I). */
size_t moe_expert_ffn_mxfp4_workspace_bytes(int rows_cap, int n_ffn, int I);
moe_status moe_expert_ffn_mxfp4(const void *x, const uint8_t *x_scales, int T, int K,
                                const int32_t *row_src, const int32_t *offsets, int rows_cap,
                                int n_ffn, int H, int I, const uint8_t *w13,
                                const uint8_t *w13_scales, const uint8_t *w2,
                                const uint8_t *w2_scales, void *y_perm, void *ws,
                                size_t ws_bytes, void *stream);

/* The norm before a block (root mean square):
 *   y[t] = x[t] / sqrt(mean over h of x[t][h]^2 + eps) * weight[h]
 * x [T][H] in x_dtype, weight [H] fp32 or NULL (ones), y [T][H] in y_dtype;
 * fp32 arithmetic; rows whose squares fp32 cannot hold are scaled by a power of
 * two first, so that finite rows of any size are normed.  y may be x when the
 * dtypes are equal.
 * MOE_ERR_SHAPE: T < 1, H < 1, H % 8, H > 32768, or eps negative or not
 * finite.  MOE_ERR_ALIGN: x, y, weight 16 bytes. */
moe_status moe_norm(const void *x, int x_dtype, const float *weight, float eps, int T, int H,
                    void *y, int y_dtype, void *stream);

/* What follows a block, in one pass: the norm of its output, the gate and
 * residual scale, the residual sum and the norm before the next block.
 *   z[t]    = norm(y[t]; w_post), or y[t] where w_post is NULL
 *   s[t][h] = residual[t][h] + scale * gate * z[t][h]          (fp32)
 *   res_out = s in res_dtype
 *   next    = norm(s; w_next) in y_dtype, taken from the fp32 sums; only
 *             where next is not NULL (w_next NULL: ones)
 * gate: none (MOE_GATE_NONE, gate NULL), gate[h] (MOE_GATE_CHANNEL, [H]) or
 * gate[t] (MOE_GATE_TOKEN, [T]), fp32.
 * y [T][H] in y_dtype, residual and res_out [T][H] in res_dtype.  res_out may
 * be residual, and next may be y; no other two may overlap.
 * A scale or gate of zero adds zero times z (a NaN in z stays one).
 * Errors as for moe_norm (every pointer 16-byte aligned, a token gate too),
 * MOE_ERR_SHAPE also for a scale that is not finite or an unknown gate kind,
 * MOE_ERR_NULL for a gate kind without a gate. */
enum { MOE_GATE_NONE = 0, MOE_GATE_CHANNEL = 1, MOE_GATE_TOKEN = 2 };
moe_status moe_norm_residual(const void *y, int y_dtype, const float *w_post, float eps,
                             const float *gate, int gate_kind, float scale, const void *residual,
                             int res_dtype, void *res_out, const float *w_next, void *next, int T,
                             int H, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_BLOCK_H */

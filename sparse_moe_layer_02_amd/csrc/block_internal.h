// Launchers of the 4-bit expert weights and the block norms (each returns
// hipGetLastError() after enqueueing).
#pragma once

#include "../../include/moe_mi355x_block.h"
#include "moe_internal.h"

namespace moe {

hipError_t launch_mxfp4_quantize(const void* x, int dtype, long long rows, int cols,
                                 const int32_t* n_rows, uint8_t* codes, uint8_t* scales,
                                 hipStream_t s);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int dtype,
                                   long long rows, int cols, void* y, hipStream_t s);

namespace mx {
// Bytes of the m-tile list in front of every workspace.
size_t tile_list_bytes(int rows_cap, int n_experts);
// Whether the products fit the launch limits (blocks of a grid).
bool grid_fits(int rows_cap, int n_experts, int N);
// rows_max: upper bound of an expert's rows.  list: the m-tile list is filled
// by launch_tiles for the same offsets, rows_cap, rows_max and form of rows.
hipError_t launch_tiles(const int32_t* offsets, int rows_cap, int n_experts, int rows_max,
                        bool fp4_rows, void* ws, hipStream_t s);
hipError_t launch_product(const void* a, const uint8_t* a_scales, const int32_t* row_src, int T,
                          int K, const int32_t* offsets, int rows_cap, int n_experts, int rows_max,
                          int D, int N, const uint8_t* w, const uint8_t* w_scales, bool swiglu,
                          int out_dtype, void* out, void* ws, hipStream_t s);
}  // namespace mx

hipError_t launch_norm(const void* x, int x_dtype, const float* weight, float eps, int T, int H,
                       void* y, int y_dtype, hipStream_t s);
hipError_t launch_norm_residual(const void* y, int y_dtype, const float* w_post, float eps,
                                const float* gate, int gate_kind, float scale,
                                const void* residual, int res_dtype, void* res_out,
                                const float* w_next, void* next, int T, int H, hipStream_t s);

}  // namespace moe

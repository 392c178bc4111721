// Grouped products of bf16 rows on MXFP4 weights (the kernels are in mx_gemm.h).
#include "mx_gemm.h"

namespace moe {
namespace mx {
MX_INSTANTIATE(false)
}  // namespace mx
}  // namespace moe

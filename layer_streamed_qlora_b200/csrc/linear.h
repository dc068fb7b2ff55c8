// Kernels of the frozen projection beside the GEMM engine.
#pragma once

#include "soup_internal.h"

namespace soup {

// y [T, out] = x [T, in] W^T, W MXFP4, 1 <= T <= MX4_FEW_TOKENS.
constexpr int MX4_FEW_TOKENS = 16;
soup_status mx4_few(const soup_weight* W, const uint16_t* x, int64_t ldx, int T, uint16_t* y, int64_t ldy,
                    cudaStream_t st);

// The same on tcgen05, for any T; trans: dx [T, in] = dy [T, out] W (x, y are dy, dx).
soup_status mx4_mid(const soup_weight* W, bool trans, const uint16_t* x, int64_t ldx, int T, uint16_t* y, int64_t ldy,
                    cudaStream_t st);

}  // namespace soup

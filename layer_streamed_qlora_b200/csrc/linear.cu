// The frozen projection without adapters: y = x W^T and its input gradient
// dx = dy W (W is frozen, so there is no weight gradient), for every storage
// of W.
//
// NF4 and bf16 weights, and MXFP4 ones with many tokens, run on the GEMM
// engine.  Its 256 x 256 tiles leave most of the GPU idle when T is small;
// with a workspace the tiles that do not fill a round are cut along K (slices
// of at least 40 k-blocks: with 16 a 2048 x 512 x 1024 product took 24.7 us in
// slices and 11.8 whole, and 1280 x 6144 x 4096, which leaves 46 tiles, 81 and
// 61), summed in slice order.  Products of 64 k-blocks are never cut then: the
// 4 tiles that 2048 x 4096 x 14336 leaves, backward, cost a round of their own.
// MXFP4 weights with fewer tokens have kernels of their own.  Forward, us in
// graph replays over weights that L2 does not hold:
//   6144 x 4096, T    1     8     16    33    64    256   512   768   1024  2048
//   mx4_few           7.6   8.1   15.8
//   mx4_mid           13.5  13.5  13.7  14.4  14.6  19.3  27.8  28.2  52.3  79.9
//   engine            33.2        32.9  33.0  33.2  33.8  34.2  34.8  62.1  89.2
//   28672 x 4096, T   1     8     16    33    64    256   512   768   1024  2048
//   mx4_few           23.9  28.2  52.2
//   mx4_mid           41.7  41.5  41.6  42.5  43.6  55.1  111   147   221   372
//   engine            75.6        60.5  60.9  61.1  62.3  113   148   200   411
// so mx4_few takes up to 8 tokens of the forward and mx4_mid up to 1024, where
// the engine is ahead for the largest matrices alone (from 800 tokens of 28672
// x 4096; backward 161 against 200 us at 768).  From 9 to 16 tokens mx4_few
// needs twice the registers and instructions, and wins only where each SM has
// one of its CTAs at most (16 rows each): at 16 tokens 13.5 us against 16.4 for
// 2048 x 11008, but 23.0 against 20.6 for 4096 x 14336.  The input gradient has
// mx4_mid from one token on (13.6 us at 6144 x 4096).
// NF4 and bf16 weights have the engine's 256-token tiles at any T: one token
// through 6144 x 4096 takes 39 and 33 us, where reading W takes 2.2 and 7.7.
#include <algorithm>

#include "gemm.h"
#include "linear.h"
#include "lora_internal.h"

namespace soup {
namespace {

constexpr int64_t MX4_MID_TOKENS = 1024;
constexpr int64_t MAX_SLICES = 148;  // two per CTA pair: 37 MiB of partials at most

size_t workspace_bytes_for(int64_t M, int64_t N) {
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  return SK_COUNTER_BYTES + (size_t)std::min<int64_t>(tiles * 8, MAX_SLICES) * SK_SLICE_BYTES;
}

soup_status check_linear(const char* fn, const soup_weight* W, const void* a, int64_t lda, int64_t a_cols, int64_t T,
                         const void* c, int64_t ldc, int64_t c_cols, const void* ws, size_t ws_bytes) {
  SOUP_TRY(check_weight(W, fn));
  SOUP_CHECK(T >= 0 && T < (1 << 30), SOUP_ERR_SHAPE, "%s: T=%lld", fn, (long long)T);
  if (T == 0) return SOUP_OK;
  SOUP_CHECK(a && c, SOUP_ERR_INVALID_ARG, "%s: null pointer", fn);
  SOUP_CHECK(lda >= a_cols && ldc >= c_cols, SOUP_ERR_SHAPE, "%s: a row stride is less than the row", fn);
  SOUP_CHECK(soup_aligned(a, 16) && soup_aligned(c, 16) && lda % 8 == 0 && ldc % 8 == 0, SOUP_ERR_ALIGN,
             "%s: rows of x, y, dy and dx must be 16-byte aligned", fn);
  SOUP_CHECK(!ws_bytes || (ws && soup_aligned(ws, 256)), SOUP_ERR_ALIGN, "%s: workspace null or not 256-byte aligned",
             fn);
  return SOUP_OK;
}

void use_workspace(GemmDesc& g, void* ws, size_t bytes) {
  if (!ws || bytes < SK_COUNTER_BYTES + 2 * SK_SLICE_BYTES) return;
  g.sk_counters = static_cast<unsigned long long*>(ws);
  g.sk_scratch = static_cast<char*>(ws) + SK_COUNTER_BYTES;
  g.sk_scratch_bytes = std::min(bytes - SK_COUNTER_BYTES, (size_t)MAX_SLICES * SK_SLICE_BYTES);
  g.sk_min_kb = 40;
}

}  // namespace
}  // namespace soup

using namespace soup;

extern "C" size_t soup_linear_workspace(const soup_weight* W, int64_t T) {
  if (!W || T <= 0 || W->out_features <= 0 || W->in_features <= 0) return 0;
  if (W->kind == SOUP_WEIGHT_MXFP4 && T <= MX4_MID_TOKENS) return 0;
  return std::max(workspace_bytes_for(T, W->out_features), workspace_bytes_for(T, W->in_features));
}

extern "C" soup_status soup_linear_fwd(const soup_weight* W, const uint16_t* x, int64_t ldx, int64_t T, uint16_t* y,
                                       int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  SOUP_TRY(check_linear("soup_linear_fwd", W, x, ldx, W ? W->in_features : 0, T, y, ldy, W ? W->out_features : 0,
                        workspace, workspace_bytes));
  if (T == 0) return SOUP_OK;
  if (W->kind == SOUP_WEIGHT_MXFP4 &&
      (T <= MX4_FEW_TOKENS / 2 || (T <= MX4_FEW_TOKENS && W->out_features <= 16 * sm_count())))
    return mx4_few(W, x, ldx, (int)T, y, ldy, static_cast<cudaStream_t>(stream));
  if (W->kind == SOUP_WEIGHT_MXFP4 && T <= MX4_MID_TOKENS)
    return mx4_mid(W, false, x, ldx, (int)T, y, ldy, static_cast<cudaStream_t>(stream));
  GemmDesc g;
  g.M = (int)T; g.N = (int)W->out_features; g.K = (int)W->in_features;
  g.A = Mat{x, T, W->in_features, ldx};
  set_weight_fwd(g, W);
  g.out_kind = OUT_BF16; g.out = y; g.ldo = ldy;
  use_workspace(g, workspace, workspace_bytes);
  return gemm(g, static_cast<cudaStream_t>(stream));
}

extern "C" soup_status soup_linear_bwd(const soup_weight* W, const uint16_t* dy, int64_t lddy, int64_t T, uint16_t* dx,
                                       int64_t lddx, void* workspace, size_t workspace_bytes, void* stream) {
  SOUP_TRY(check_linear("soup_linear_bwd", W, dy, lddy, W ? W->out_features : 0, T, dx, lddx, W ? W->in_features : 0,
                        workspace, workspace_bytes));
  if (T == 0) return SOUP_OK;
  if (W->kind == SOUP_WEIGHT_MXFP4 && T <= MX4_MID_TOKENS)
    return mx4_mid(W, true, dy, lddy, (int)T, dx, lddx, static_cast<cudaStream_t>(stream));
  GemmDesc g;
  g.M = (int)T; g.N = (int)W->in_features; g.K = (int)W->out_features;
  g.A = Mat{dy, T, W->out_features, lddy};
  set_weight_bwd(g, W);
  g.out_kind = OUT_BF16; g.out = dx; g.ldo = lddx;
  use_workspace(g, workspace, workspace_bytes);
  return gemm(g, static_cast<cudaStream_t>(stream));
}

// MXFP4 block quantisation (shard building) and standalone dequantisation.
//
// Quantise, per block of 32: the scale exponent is e = floor(log2 amax) - 2
// (2 = the exponent of E2M1's largest value, 6), at least -127: with E the
// fp32 exponent field of amax, the scale byte is max(E - 2, 0).  A code is
// the E2M1 value nearest to w 2^-e (exact in fp32 but for parts far below
// half the smallest step), ties to even, saturating at 6.  The block maximum
// is taken on the bit patterns of |w|, where NaN and infinity rank above
// every finite value, so one comparison finds a non-finite block.
#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "mx4.cuh"
#include "ptx.cuh"
#include "soup_internal.h"

namespace soup {
namespace {

// 32 bytes: one access where aligned (v32), else two of 16.
__device__ __forceinline__ void load_32B(const void* p, uint32_t (&w)[8], bool v32) {
  if (v32) {
    ptx::ld_global_32B(p, w);
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void store_32B(void* p, const uint32_t (&w)[8], bool v32) {
  if (v32) {
    ptx::st_global_32B(p, w);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Both kernels are bound by HBM: one thread per 16 elements (half a block),
// whose loads and stores are 8 to 64 bytes each.  28672 x 4096 fp32 quantise
// in 112 us (6.9 TB/s; with 8 elements per thread 134), 4096 x 14336 dequantise
// in 24.0 (6.2 TB/s; 28.8, and 26.6 without the early launch).  `dense`: scale
// rows have no padding (in a multiple of 512), so a block's index is its
// scale's and no division by the row length is needed; `packed` the same for
// W's rows.
// W, codes and scales are read by ordinary loads: see dependent_launch.
template <bool BF16>
__global__ void __launch_bounds__(256)
    mx4_quantize_kernel(const void* W, int64_t units, uint32_t units_per_row, int64_t ldw, uint2* codes,
                        uint8_t* scales, int64_t scale_stride, uint8_t* values, bool v32_in, bool v32_out, bool dense,
                        bool packed, int32_t* nonfinite) {
  ptx::grid_dep_wait();
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool in_range = u < units;  // the same for both halves of a block
  uint32_t row = 0, c = 0;
  if (!(dense && packed) && in_range) {
    row = (uint32_t)(u / units_per_row);
    c = (uint32_t)(u - (int64_t)row * units_per_row);
  }
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
  if (in_range) {
    const int64_t at = packed ? u * 16 : row * ldw + c * (int64_t)16;
    if (BF16) {
      uint32_t w[8];
      load_32B(static_cast<const uint16_t*>(W) + at, w, v32_in);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      uint32_t w0[8], w1[8];
      load_32B(static_cast<const float*>(W) + at, w0, v32_in);
      load_32B(static_cast<const float*>(W) + at + 8, w1, v32_in);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __uint_as_float(w0[i]);
        x[8 + i] = __uint_as_float(w1[i]);
      }
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  if (!in_range) return;
  const uint32_t E = top >> 23;
  const bool bad = E == 255;
  const uint32_t s = bad ? 255u : (E > 2 ? E - 2 : 0u);
  const float up = __uint_as_float((254u - (bad ? 0u : s)) << 23);  // 2^(127 - s)
  uint32_t code[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    code[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(x[2 * i] * up, x[2 * i + 1] * up), __NV_E2M1,
                                                       cudaRoundNearest)
                    << (8 * (i & 3));
  if (bad) code[0] = code[1] = 0;
  codes[u] = make_uint2(code[0], code[1]);
  if ((u & 1) == 0) {
    scales[dense ? u >> 1 : row * scale_stride + (c >> 1)] = (uint8_t)s;
    if (bad && nonfinite) *nonfinite = 1;
  }
  // the bytes that pad a row of scales
  if (!dense && c == units_per_row - 1)
    for (int64_t p = units_per_row / 2; p < scale_stride; ++p) scales[row * scale_stride + p] = 0;
  if (values) {
    uint32_t o[8];
    mx4_decode<2>(code, s, o);
    store_32B(values + u * 32, o, v32_out);
  }
}

__global__ void __launch_bounds__(256)
    mx4_dequant_kernel(const uint2* codes, const uint8_t* scales, int64_t units, uint32_t units_per_row,
                       int64_t scale_stride, uint8_t* out, bool v32, bool dense) {
  ptx::grid_dep_wait();
  const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (u >= units) return;
  const uint2 c = codes[u];
  int64_t at = u >> 1;
  if (!dense) {
    const uint32_t row = (uint32_t)(u / units_per_row);
    at = row * scale_stride + ((u - (int64_t)row * units_per_row) >> 1);
  }
  const uint32_t w[2] = {c.x, c.y};
  uint32_t o[8];
  mx4_decode<2>(w, scales[at], o);
  store_32B(out + u * 32, o, v32);
}

soup_status mx4_check_shape(const char* fn, int64_t out, int64_t in) {
  SOUP_CHECK(out > 0 && in > 0 && in % 32 == 0, SOUP_ERR_SHAPE,
             "%s: need out > 0 and in a positive multiple of 32 (out=%lld in=%lld)", fn, (long long)out, (long long)in);
  // at most 2^31 - 1 blocks of 256 threads with 16 elements each
  SOUP_CHECK(out < (1ll << 30) && in < (1ll << 30) && out * (in / 16) < 255ll << 31, SOUP_ERR_SHAPE,
             "%s: %lld x %lld is too large", fn, (long long)out, (long long)in);
  return SOUP_OK;
}

}  // namespace
}  // namespace soup

using namespace soup;

extern "C" int64_t soup_mx4_scale_stride(int64_t in) { return in > 0 ? mx4_scale_stride(in) : 0; }

extern "C" soup_status soup_mx4_quantize(const void* W, int32_t w_type, int64_t out, int64_t in, int64_t ldw,
                                         uint8_t* codes, uint8_t* scales, uint16_t* W_bf16, int32_t* nonfinite_dev,
                                         void* stream) {
  SOUP_CHECK(W && codes && scales, SOUP_ERR_INVALID_ARG, "soup_mx4_quantize: null pointer");
  SOUP_CHECK(w_type == SOUP_TYPE_F32 || w_type == SOUP_TYPE_BF16, SOUP_ERR_INVALID_ARG,
             "soup_mx4_quantize: w_type %d is neither SOUP_TYPE_F32 nor SOUP_TYPE_BF16", w_type);
  SOUP_TRY(mx4_check_shape("soup_mx4_quantize", out, in));
  SOUP_CHECK(ldw >= in, SOUP_ERR_SHAPE, "soup_mx4_quantize: ldw %lld < in", (long long)ldw);
  const int es = w_type == SOUP_TYPE_F32 ? 4 : 2;
  SOUP_CHECK(soup_aligned(W, 16) && (ldw * es) % 16 == 0 && soup_aligned(codes, 16) && soup_aligned(scales, 16) &&
                 soup_aligned(W_bf16, 16) && soup_aligned(nonfinite_dev, 4),
             SOUP_ERR_ALIGN,
             "soup_mx4_quantize: W, its rows, codes, scales and W_bf16 must be 16-byte aligned, the flag 4-byte");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const uint32_t upr = (uint32_t)(in / 16);
  const int64_t units = out * (in / 16), ss = mx4_scale_stride(in);
  const unsigned grid = (unsigned)((units + 255) / 256);
  const bool v32_in = soup_aligned(W, 32) && (ldw * es) % 32 == 0, v32_out = soup_aligned(W_bf16, 32);
  const bool dense = ss == in / 32, packed = ldw == in || out == 1;
  uint2* c = reinterpret_cast<uint2*>(codes);
  uint8_t* v = reinterpret_cast<uint8_t*>(W_bf16);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = dependent_launch(grid, 256, 0, st, attr);
  SOUP_CUDA_TRY(cudaLaunchKernelEx(&cfg, w_type == SOUP_TYPE_BF16 ? mx4_quantize_kernel<true> : mx4_quantize_kernel<false>,
                                   W, units, upr, ldw, c, scales, ss, v, v32_in, v32_out, dense, packed,
                                   nonfinite_dev));
  SOUP_LAUNCH_CHECK();
  return SOUP_OK;
}

extern "C" soup_status soup_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t out, int64_t in,
                                        uint16_t* W_bf16, void* stream) {
  SOUP_CHECK(codes && scales && W_bf16, SOUP_ERR_INVALID_ARG, "soup_mx4_dequant: null pointer");
  SOUP_TRY(mx4_check_shape("soup_mx4_dequant", out, in));
  SOUP_CHECK(soup_aligned(codes, 16) && soup_aligned(scales, 16) && soup_aligned(W_bf16, 16), SOUP_ERR_ALIGN,
             "soup_mx4_dequant: codes, scales and W_bf16 must be 16-byte aligned");
  const int64_t units = out * (in / 16), ss = mx4_scale_stride(in);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      dependent_launch((unsigned)((units + 255) / 256), 256, 0, static_cast<cudaStream_t>(stream), attr);
  SOUP_CUDA_TRY(cudaLaunchKernelEx(&cfg, mx4_dequant_kernel, reinterpret_cast<const uint2*>(codes), scales, units,
                                   (uint32_t)(in / 16), ss, reinterpret_cast<uint8_t*>(W_bf16),
                                   (bool)soup_aligned(W_bf16, 32), ss == in / 32));
  SOUP_LAUNCH_CHECK();
  return SOUP_OK;
}

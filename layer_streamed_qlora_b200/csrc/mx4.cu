// MXFP4 block quantisation (shard building) and standalone dequantisation.
//
// Quantise, per block of 32: the scale exponent is e = floor(log2 amax) - 2
// (2 = the exponent of E2M1's largest value, 6), at least -127: with E the
// fp32 exponent field of amax, the scale byte is max(E - 2, 0).  A code is
// the E2M1 value nearest to w 2^-e (exact in fp32 but for parts far below
// half the smallest step), ties to even, saturating at 6.  The block maximum
// is taken on the bit patterns of |w|, where NaN and infinity rank above
// every finite value, so one comparison finds a non-finite block.
#include <algorithm>

#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include "mx4.cuh"
#include "ptx.cuh"
#include "soup_internal.h"

namespace soup {
namespace {

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// One thread per 8 elements; the 4 threads of a block share its maximum.
template <bool BF16>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const void* __restrict__ W, uint32_t units,
                                                           uint32_t units_per_row, int64_t ldw,
                                                           uint32_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                           int64_t scale_stride, uint4* __restrict__ values,
                                                           int32_t* __restrict__ nonfinite) {
  // warps run the loop together (the shuffles want all lanes); units is a
  // multiple of 4, so the 4 lanes of a block are in range or not together
  const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
  for (uint64_t u0 = (uint64_t)blockIdx.x * blockDim.x + (threadIdx.x & ~31u); u0 < units; u0 += stride) {
    const uint64_t u64 = u0 + (threadIdx.x & 31);
    const bool in_range = u64 < units;
    const uint32_t u = in_range ? (uint32_t)u64 : 0u;
    const uint32_t row = u / units_per_row, c = u - row * units_per_row;
    float x[8];
    if (BF16) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + row * ldw + 8 * (int64_t)c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + row * ldw + 8 * (int64_t)c);
      const float4 a = p[0], b = p[1];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (!in_range) continue;
    const uint32_t E = top >> 23;
    const bool bad = E == 255;
    const uint32_t s = bad ? 255u : (E > 2 ? E - 2 : 0u);
    const float up = __uint_as_float((254u - (bad ? 0u : s)) << 23);  // 2^(127 - s)
    uint32_t code = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      code |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(x[2 * i] * up, x[2 * i + 1] * up), __NV_E2M1,
                                                 cudaRoundNearest)
              << (8 * i);
    if (bad) code = 0;
    codes[u] = code;
    if ((c & 3) == 0) {
      scales[row * scale_stride + (c >> 2)] = (uint8_t)s;
      if (bad && nonfinite) *nonfinite = 1;
    }
    // the bytes that pad a row of scales
    if (c == units_per_row - 1)
      for (int64_t p = units_per_row / 4; p < scale_stride; ++p) scales[row * scale_stride + p] = 0;
    if (values) {
      uint32_t o[4];
      mx4_decode<1>(&code, s, o);
      values[u] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// One thread per 8 codes.
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const uint32_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ scales, uint32_t units,
                                                          uint32_t units_per_row, int64_t scale_stride,
                                                          uint4* __restrict__ out) {
  const uint32_t stride = gridDim.x * blockDim.x;
  for (uint64_t u64 = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; u64 < units; u64 += stride) {
    const uint32_t u = (uint32_t)u64;
    const uint32_t row = u / units_per_row, c = u - row * units_per_row;
    uint32_t o[4];
    const uint32_t w = codes[u];
    mx4_decode<1>(&w, scales[row * scale_stride + (c >> 2)], o);
    out[u] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

soup_status mx4_check_shape(const char* fn, int64_t out, int64_t in) {
  SOUP_CHECK(out > 0 && in > 0 && in % 32 == 0, SOUP_ERR_SHAPE,
             "%s: need out > 0 and in a positive multiple of 32 (out=%lld in=%lld)", fn, (long long)out, (long long)in);
  SOUP_CHECK(out < (1ll << 30) && in < (1ll << 30) && out * (in / 8) < (1ll << 32), SOUP_ERR_SHAPE,
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
  const uint32_t upr = (uint32_t)(in / 8), units = (uint32_t)(out * (in / 8));
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)units + 255) / 256, (int64_t)sm_count() * 16);
  const int64_t ss = mx4_scale_stride(in);
  uint4* v = reinterpret_cast<uint4*>(W_bf16);
  if (w_type == SOUP_TYPE_BF16)
    mx4_quantize_kernel<true><<<grid, 256, 0, st>>>(W, units, upr, ldw, reinterpret_cast<uint32_t*>(codes), scales, ss,
                                                    v, nonfinite_dev);
  else
    mx4_quantize_kernel<false><<<grid, 256, 0, st>>>(W, units, upr, ldw, reinterpret_cast<uint32_t*>(codes), scales,
                                                     ss, v, nonfinite_dev);
  SOUP_LAUNCH_CHECK();
  return SOUP_OK;
}

extern "C" soup_status soup_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t out, int64_t in,
                                        uint16_t* W_bf16, void* stream) {
  SOUP_CHECK(codes && scales && W_bf16, SOUP_ERR_INVALID_ARG, "soup_mx4_dequant: null pointer");
  SOUP_TRY(mx4_check_shape("soup_mx4_dequant", out, in));
  SOUP_CHECK(soup_aligned(codes, 16) && soup_aligned(scales, 16) && soup_aligned(W_bf16, 16), SOUP_ERR_ALIGN,
             "soup_mx4_dequant: codes, scales and W_bf16 must be 16-byte aligned");
  const uint32_t upr = (uint32_t)(in / 8), units = (uint32_t)(out * (in / 8));
  const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)units + 255) / 256, (int64_t)sm_count() * 16);
  mx4_dequant_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<const uint32_t*>(codes), scales, units, upr, mx4_scale_stride(in),
      reinterpret_cast<uint4*>(W_bf16));
  SOUP_LAUNCH_CHECK();
  return SOUP_OK;
}

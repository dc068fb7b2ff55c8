// MXFP4 (OCP microscaling) storage of the frozen base: blocks of 32
// consecutive elements along `in`, each element E2M1 (sign, 2 exponent bits,
// 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), one E8M0 scale byte s per
// block standing for 2^(s - 127) (255: NaN).  Byte j of a row holds element
// 2j in bits 3..0 and 2j + 1 in bits 7..4.  A row of scales is padded to a
// multiple of 16 bytes, so that TMA can stage any row length.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace soup {

__host__ __device__ constexpr int64_t mx4_scale_stride(int64_t in) { return (in / 32 + 15) / 16 * 16; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A code's exponent and mantissa bits moved to bits 8..6 of a bf16 are the
// element times 2^-126 (code exponent 0 lands on a bf16 subnormal, which has
// the same meaning), so that times 2^(s - 1) is the stored value; the product
// is exact (two significant bits) down to bf16's smallest subnormal.  2^(s -
// 1) is a bf16 up to s = 128 (scales up to 2); above, the rest of it follows
// in a second product (mx4_large), where a value beyond bf16's largest
// becomes infinite and s = 255 gives NaN.
__device__ __forceinline__ uint32_t mx4_scale_bf16x2(uint32_t s) { return (min(s, 128u) + 126u) * 0x00800080u; }
__device__ __forceinline__ bool mx4_is_large(uint32_t s) { return s > 128; }
__device__ __forceinline__ uint32_t mx4_large_bf16x2(uint32_t s) {
  return s == 255 ? 0x7FC07FC0u : (s - 1u) * 0x00800080u;  // 2^(s - 128)
}

// 8 codes (one word, element k in bits 4k..4k+3) times `scale2` as 4 bf16x2
// words in element order.  A product with two powers of two makes two copies
// of a byte at once: the masks then find both codes' exponents and mantissas
// (copies 6 and 18 up) and both signs (12 and 24 up) in place, without
// permutes, and half of the work is the multiplier's.  (With shifts for pairs
// (k, k + 4) and permutes after, the decode was bound by the integer pipe.)
__device__ __forceinline__ void mx4_decode8_scaled(uint32_t w, uint32_t scale2, uint32_t* o) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = __byte_perm(w, 0, 0x4440 + j);
    o[j] = mul_bf16x2(((b * 0x00040040u) & 0x01C001C0u) | ((b * 0x01001000u) & 0x80008000u), scale2);
  }
}

// N words of one block (scale byte s).
template <int N>
__device__ __forceinline__ void mx4_decode(const uint32_t* w, uint32_t s, uint32_t* o) {
  const uint32_t scale2 = mx4_scale_bf16x2(s);
#pragma unroll
  for (int u = 0; u < N; ++u) mx4_decode8_scaled(w[u], scale2, o + 4 * u);
  if (mx4_is_large(s)) {
    const uint32_t more = mx4_large_bf16x2(s);
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) o[i] = mul_bf16x2(o[i], more);
  }
}

}  // namespace soup

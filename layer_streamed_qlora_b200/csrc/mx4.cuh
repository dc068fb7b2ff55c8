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

// bf16x2 with 2^(s - 127) in both halves: the exponent field is s itself;
// s = 0 is the subnormal 2^-127 and s = 255 a NaN.
__device__ __forceinline__ uint32_t mx4_scale_bf16x2(uint32_t s) {
  const uint32_t h = s == 0 ? 0x0040u : (s == 255 ? 0x7FC0u : s << 7);
  return h * 0x00010001u;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 8 codes (one word, element k in bits 4k..4k+3) times the block scale, as 4
// bf16x2 words in element order.  A code's exponent and mantissa bits moved
// to bits 8..6 of a bf16 are the value times 2^-126 (code exponent 0 lands
// on a bf16 subnormal, which has the same meaning), so one multiplication by
// 2^126 gives the element, and one by the scale the stored value; both are
// exact (the value has two significant bits) down to bf16's smallest
// subnormal, and a value beyond bf16's largest becomes infinite.  Elements k
// and k + 4 share a word until the permutes put neighbours together.
__device__ __forceinline__ void mx4_decode8(uint32_t w, uint32_t scale2, uint32_t (&o)[4]) {
  constexpr uint32_t MAG = 0x01C001C0u, SGN = 0x80008000u, UP = 0x7E807E80u;  // UP: 2^126
  uint32_t p0 = ((w << 6) & MAG) | ((w << 12) & SGN);
  uint32_t p1 = ((w << 2) & MAG) | ((w << 8) & SGN);
  uint32_t p2 = ((w >> 2) & MAG) | ((w << 4) & SGN);
  uint32_t p3 = ((w >> 6) & MAG) | (w & SGN);
  p0 = mul_bf16x2(mul_bf16x2(p0, UP), scale2);
  p1 = mul_bf16x2(mul_bf16x2(p1, UP), scale2);
  p2 = mul_bf16x2(mul_bf16x2(p2, UP), scale2);
  p3 = mul_bf16x2(mul_bf16x2(p3, UP), scale2);
  o[0] = __byte_perm(p0, p1, 0x5410);
  o[1] = __byte_perm(p2, p3, 0x5410);
  o[2] = __byte_perm(p0, p1, 0x7632);
  o[3] = __byte_perm(p2, p3, 0x7632);
}

}  // namespace soup

// AdamW over a group of tensors in one launch, optimiser states in fp32 or in
// MXFP8 (8-bit elements, one E8M0 scale byte per block of 32): E4M3 for m,
// E5M2 for v, whose range is squared.
//
// The update has the formula of optim.cu, but its root and quotient are not
// correctly rounded ones (see below).  With 8-bit states a step decodes m and v
// of each element, forms the new ones in fp32, updates theta from these, and
// stores them again, each rounded to one of its two neighbours at random with
// the probability that keeps the mean.  Rounded to nearest neither would
// follow its average: a step moves v by a part 1 - beta2 (1e-3) of itself and
// m by 1 - beta1 (0.1) of its distance from the gradient, while half a code
// step is 6 to 12 % of v and 3 to 6 % of m: v would never fall, and m would
// stop at two thirds of a constant gradient.  A v above zero keeps at least
// the smallest code, so m / sqrt(v) has no zero divisor that the fp32 state
// would not have.
// The block's scale brings the largest element to [2^7, 2^8) (E4M3) or
// [2^14, 2^15) (E5M2), below the largest value even after rounding up;
// elements of m down to 2^-17 and of v down to 2^-31 of it have a code.  An
// element that is not finite is stored as NaN and does not take part in the
// maximum.
//
// The random bits are a hash of (seed, step, tensor, element), so a step gives
// the same bits on every run and with any launch shape; m and v of an element
// share them (each rounding is unbiased by itself, and m / sqrt(v) errs less
// when both go the same way).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <exception>
#include <vector>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"
#include "soup_internal.h"

namespace soup {
namespace {

constexpr int CHUNK = 2048;  // elements per CTA turn: 256 threads x 8

// Device tables of a group: GroupTensor[n_tensors], then GroupChunk[n_chunks].
struct GroupTensor {
  int64_t n;
  float* theta;
  uint16_t* theta_bf16;
  void* grad;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  int64_t v32;  // 1: theta, grad, m and v are 32-byte aligned
};
struct GroupChunk {
  uint32_t tensor, chunk;
};

struct GroupArgs {
  const GroupTensor* tensors;
  const GroupChunk* chunks;
  int64_t n_chunks;
  float decay, beta1, one_minus_beta1, beta2, one_minus_beta2, step_size, inv_sqrt_bc2, eps, grad_scale;
  int zero_grad, tiny_eps;
  uint32_t seed, t;
  int32_t* nonfinite;
};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; }

// A bijective 32-bit mix (xor-shifts and odd multipliers, Appleby 2011).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

__device__ __forceinline__ float e8m0(uint32_t s) { return __uint_as_float(s ? s << 23 : 1u << 22); }

// The two element formats: MANT mantissa bits, exponent bias, and the
// exponent TOP that a block's largest element is brought to.
struct E4M3 {
  static constexpr uint32_t MANT = 3, BIAS = 7, TOP = 7;
};
struct E5M2 {
  static constexpr uint32_t MANT = 2, BIAS = 15, TOP = 14;
};

// Scale byte of a block whose largest magnitude has the bits `top`, and the
// factor 2^(127 - s) that brings the block to the format's range.
template <class F>
__device__ __forceinline__ uint32_t block_scale(uint32_t top, float& up) {
  const uint32_t E = top >> 23, s = E > F::TOP ? E - F::TOP : 0u;
  up = __uint_as_float((254u - s) << 23);
  return s;
}

// Codes 2 * pair and 2 * pair + 1 of a word of four.  E5M2 is the upper byte
// of an fp16.
__device__ __forceinline__ float2 e4m3_pair(uint32_t w, int pair) {
  const uint16_t c = (uint16_t)(pair ? w >> 16 : w);
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
}
__device__ __forceinline__ float2 e5m2_pair(uint32_t w, int pair) {
  const uint32_t h = __byte_perm(w, 0, pair ? 0x3424 : 0x1404);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Magnitude code of y in [0, 2^(TOP + 1)), the dropped mantissa bits rounded
// by 16 random bits at their top (`rnd` holds them there, zeros elsewhere).
// Times 2^(BIAS - 127) the format's exponents are fp32's, its subnormal
// elements fp32 subnormals, and the code is the upper bits of the fp32.
template <class F>
__device__ __forceinline__ uint32_t encode_stochastic(float y, uint32_t rnd) {
  constexpr float TO_BIAS = F::BIAS == 7 ? 0x1p-120f : 0x1p-112f;
  static_assert(F::BIAS == 7 || F::BIAS == 15, "2^(BIAS - 127)");
  return (__float_as_uint(y * TO_BIAS) + rnd) >> (23 - F::MANT);
}

// The low bytes of four words in one.
__device__ __forceinline__ uint32_t pack_bytes(const uint32_t* c) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

// Special-function approximations (subnormal arguments and results as 0).
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
  return d;
}

__device__ __forceinline__ float new_m(const GroupArgs& a, float m, float g) {
  return __fadd_rn(__fmul_rn(m, a.beta1), __fmul_rn(g, a.one_minus_beta1));
}
__device__ __forceinline__ float new_v(const GroupArgs& a, float v, float g) {
  return __fadd_rn(__fmul_rn(v, a.beta2), __fmul_rn(__fmul_rn(g, g), a.one_minus_beta2));
}

// 8 fp32 values: 32-byte accesses where v32 (p 32-byte aligned), else 16-byte.
__device__ __forceinline__ void load8(const float* p, float (&x)[8], bool v32) {
  if (v32) {
    uint32_t w[8];
    ptx::ld_global_32B(p, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8], bool v32) {
  if (v32) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[i]);
    ptx::st_global_32B(p, w);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// The bits of the largest finite |x| over a block of 32 (4 lanes of 8); odd:
// some element of this thread's is not finite.
__device__ __forceinline__ uint32_t block_top(const float (&x)[8], bool& odd) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_abs_nan(top, x[i]);
  odd = !finite(top);
  if (odd) {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (finite(x[i])) top = fmaxf(top, fabsf(x[i]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  return __float_as_uint(fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2)));
}

// One thread per 8 elements of a chunk: 4 lanes share a block of 32, and all
// of a tensor's arrays move in 8- to 32-byte accesses.  41.9 M parameters take
// 145 to 151 us with 8-bit states and fp32 gradients (5.0 to 5.2 TB/s: 72
// instructions per element keep 60 % of the issue slots busy), 138 with bf16
// gradients (the same instructions for fewer bytes), and 181 to 183 us with
// fp32 states and bf16 gradients (6.4 TB/s, the copy rate); five CTAs per SM
// spill, and are slower (164, 199).  1.3 M parameters (640 chunks) are a round
// of the 592 resident CTAs and 48 CTAs more: 7.3 us from L2.  The elements
// beyond a tensor's end (in its last chunk alone) count as zeros and are not
// stored.
template <int BITS, bool G16>
__global__ void __launch_bounds__(256, 4) adamw_group_kernel(const GroupArgs a) {
  ptx::grid_dep_wait();
  bool bad = false;
  for (int64_t c = blockIdx.x; c < a.n_chunks; c += gridDim.x) {
    const GroupChunk ch = a.chunks[c];
    const GroupTensor t = a.tensors[ch.tensor];
    const int64_t i0 = (int64_t)ch.chunk * CHUNK + threadIdx.x * 8;
    const int64_t left = t.n - i0;
    const int in = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    const bool v32 = t.v32;
    float p[8], g[8], m[8], v[8];
    if (in == 8) {
      load8(t.theta + i0, p, v32);
      if (G16) {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(t.grad) + i0);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[2 * i] = __uint_as_float(ws[i] << 16);
          g[2 * i + 1] = __uint_as_float(ws[i] & 0xFFFF0000u);
        }
      } else {
        load8(static_cast<const float*>(t.grad) + i0, g, v32);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool ok = i < in;
        p[i] = ok ? t.theta[i0 + i] : 0.f;
        if (G16) g[i] = ok ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.grad)[i0 + i]) : 0.f;
        else g[i] = ok ? static_cast<const float*>(t.grad)[i0 + i] : 0.f;
      }
    }
    if (BITS == 32) {
      const float *ms = static_cast<const float*>(t.m) + i0, *vs = static_cast<const float*>(t.v) + i0;
      if (in == 8) {
        load8(ms, m, v32);
        load8(vs, v, v32);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m[i] = i < in ? ms[i] : 0.f;
          v[i] = i < in ? vs[i] : 0.f;
        }
      }
    } else {
      const uint8_t *ms = static_cast<const uint8_t*>(t.m) + i0, *vs = static_cast<const uint8_t*>(t.v) + i0;
      uint32_t mw[2] = {0, 0}, vw[2] = {0, 0};
      float sm = 0.f, sv = 0.f;
      if (in == 8) {
        const uint2 x = *reinterpret_cast<const uint2*>(ms), y = *reinterpret_cast<const uint2*>(vs);
        mw[0] = x.x; mw[1] = x.y; vw[0] = y.x; vw[1] = y.y;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= in) break;
          mw[i >> 2] |= (uint32_t)ms[i] << (8 * (i & 3));
          vw[i >> 2] |= (uint32_t)vs[i] << (8 * (i & 3));
        }
      }
      if (in > 0) {
        sm = e8m0(t.m_scale[i0 >> 5]);
        sv = e8m0(t.v_scale[i0 >> 5]);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 x = e4m3_pair(mw[i >> 2], (i >> 1) & 1), y = e5m2_pair(vw[i >> 2], (i >> 1) & 1);
        m[i] = x.x * sm;
        m[i + 1] = x.y * sm;
        v[i] = y.x * sv;
        v[i + 1] = y.y * sv;
      }
    }
    float gtop = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      gtop = max_abs_nan(gtop, g[i]);
      const float gi = g[i] * a.grad_scale;
      m[i] = new_m(a, m[i], gi);
      v[i] = new_v(a, v[i], gi);
      // quotient and root to a few fp32 steps (2^-21 of the update in all).  Correctly rounded ones
      // made the 8-bit step bound by instructions, 197 instead of 165 us for 41.9 M parameters, and
      // cost the 32-bit one 187 instead of 181 (flat buffers, bf16 gradients, back-to-back calls).
      // sqrt takes a subnormal v (root below 1.1e-19) as 0: times inv_sqrt_bc2 that is 2^-23 of the
      // least eps allowed on this path.
      const float q = a.tiny_eps ? __fdiv_rn(m[i], __fsqrt_rn(v[i]) * a.inv_sqrt_bc2 + a.eps)
                                 : m[i] * rcp_approx(fmaf(sqrt_approx(v[i]), a.inv_sqrt_bc2, a.eps));
      p[i] = fmaf(-a.step_size, q, p[i] * a.decay);
    }
    bad |= !finite(gtop);
    if (in == 8) {
      store8(t.theta + i0, p, v32);
      if (t.theta_bf16) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
        *reinterpret_cast<uint4*>(t.theta_bf16 + i0) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      if (a.zero_grad) {
        if (G16) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.grad) + i0) = make_uint4(0, 0, 0, 0);
        } else {
          const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          store8(static_cast<float*>(t.grad) + i0, z, v32);
        }
      }
      if (BITS == 32) {
        store8(static_cast<float*>(t.m) + i0, m, v32);
        store8(static_cast<float*>(t.v) + i0, v, v32);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= in) break;
        t.theta[i0 + i] = p[i];
        if (t.theta_bf16) t.theta_bf16[i0 + i] = (uint16_t)(pack_bf16x2(p[i], 0.f) & 0xFFFFu);
        if (a.zero_grad) {
          if (G16) static_cast<uint16_t*>(t.grad)[i0 + i] = 0;
          else static_cast<float*>(t.grad)[i0 + i] = 0.f;
        }
        if (BITS == 32) {
          static_cast<float*>(t.m)[i0 + i] = m[i];
          static_cast<float*>(t.v)[i0 + i] = v[i];
        }
      }
    }
    if (BITS == 8) {
      const uint32_t key = mix32(mix32(ch.tensor + 0x9E3779B9u * a.t) + a.seed);
      bool odd_m, odd_v;
      float um, uv;
      const uint32_t sm = block_scale<E4M3>(block_top(m, odd_m), um);
      const uint32_t sv = block_scale<E5M2>(block_top(v, odd_v), uv);
      uint32_t cm[8], cv[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const uint32_t h = mix32((uint32_t)((i0 + i) >> 1) + key);
        // 16 random bits each at the top of the 20 (E4M3) or 21 (E5M2) dropped ones
        const uint32_t r0 = (h << 4) & 0xFFFF0u, r1 = (h >> 12) & 0xFFFF0u;
        cm[i] = encode_stochastic<E4M3>(fabsf(m[i]) * um, r0);
        cm[i + 1] = encode_stochastic<E4M3>(fabsf(m[i + 1]) * um, r1);
        cv[i] = encode_stochastic<E5M2>(v[i] * uv, r0 << 1);
        cv[i + 1] = encode_stochastic<E5M2>(v[i + 1] * uv, r1 << 1);
      }
      uint32_t mw[2], vw[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float* x = m + 4 * k;
        const uint32_t sign = __byte_perm(__byte_perm(__float_as_uint(x[0]), __float_as_uint(x[1]), 0x0073),
                                          __byte_perm(__float_as_uint(x[2]), __float_as_uint(x[3]), 0x0073), 0x5410);
        mw[k] = pack_bytes(cm + 4 * k) | (sign & 0x80808080u);
        vw[k] = pack_bytes(cv + 4 * k);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // a byte 0 becomes 1 where v is above zero: the top bit of (bits of v) - 1 says where it is not
        const uint32_t zero = (vw[k] - 0x01010101u) & ~vw[k] & 0x80808080u;
        if (zero) {
          uint32_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = (__float_as_uint(v[4 * k + i]) - 1u) >> 24;
          vw[k] |= (zero & ~pack_bytes(b)) >> 7;
        }
      }
      if (odd_m || odd_v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int at = 8 * (i & 3);
          if (!finite(m[i])) mw[i >> 2] = (mw[i >> 2] & ~(0xFFu << at)) | (0x7Fu << at);
          if (!finite(v[i])) vw[i >> 2] = (vw[i >> 2] & ~(0xFFu << at)) | (0x7Fu << at);
        }
      }
      uint8_t *ms = static_cast<uint8_t*>(t.m) + i0, *vs = static_cast<uint8_t*>(t.v) + i0;
      if (in == 8) {
        *reinterpret_cast<uint2*>(ms) = make_uint2(mw[0], mw[1]);
        *reinterpret_cast<uint2*>(vs) = make_uint2(vw[0], vw[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i >= in) break;
          ms[i] = (uint8_t)(mw[i >> 2] >> (8 * (i & 3)));
          vs[i] = (uint8_t)(vw[i >> 2] >> (8 * (i & 3)));
        }
      }
      if ((threadIdx.x & 3) == 0 && in > 0) {
        t.m_scale[i0 >> 5] = (uint8_t)sm;
        t.v_scale[i0 >> 5] = (uint8_t)sv;
      }
    }
  }
  if (bad && a.nonfinite) *a.nonfinite = 1;
}

size_t align16(size_t v) { return (v + 15) / 16 * 16; }

int64_t chunks_of(int64_t n) { return (n + CHUNK - 1) / CHUNK; }

}  // namespace
}  // namespace soup

using namespace soup;

extern "C" size_t soup_adamw_group_bytes(const soup_adamw_tensor* tensors, int32_t n_tensors) {
  if (!tensors || n_tensors <= 0) return 0;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n_tensors; ++i) chunks += tensors[i].n > 0 ? chunks_of(tensors[i].n) : 0;
  return align16((size_t)n_tensors * sizeof(GroupTensor)) + (size_t)chunks * sizeof(GroupChunk);
}

extern "C" soup_status soup_adamw_group_init(const soup_adamw_tensor* tensors, int32_t n_tensors, int32_t state_bits,
                                             int32_t grad_type, void* tables_dev, size_t tables_bytes,
                                             soup_adamw_group* group, void* stream) {
  const char* fn = "soup_adamw_group_init";
  SOUP_CHECK(tensors && group, SOUP_ERR_INVALID_ARG, "%s: null pointer", fn);
  SOUP_CHECK(n_tensors >= 1, SOUP_ERR_SHAPE, "%s: n_tensors %d", fn, n_tensors);
  SOUP_CHECK(state_bits == 8 || state_bits == 32, SOUP_ERR_INVALID_ARG, "%s: state_bits %d is neither 8 nor 32", fn,
             state_bits);
  SOUP_CHECK(grad_type == SOUP_TYPE_F32 || grad_type == SOUP_TYPE_BF16, SOUP_ERR_INVALID_ARG,
             "%s: grad_type %d is neither SOUP_TYPE_F32 nor SOUP_TYPE_BF16", fn, grad_type);
  try {
    std::vector<GroupTensor> gt(n_tensors);
    std::vector<GroupChunk> gc;
    int64_t total = 0;
    struct Range {
      const char *lo, *hi;
      int32_t tensor;
    };
    std::vector<Range> ranges;
    for (int32_t i = 0; i < n_tensors; ++i) {
      const soup_adamw_tensor& s = tensors[i];
      SOUP_CHECK(s.n >= 0 && s.n < (1ll << 40), SOUP_ERR_SHAPE, "%s: tensor %d has n = %lld", fn, i, (long long)s.n);
      memset(&gt[i], 0, sizeof(gt[i]));
      if (s.n == 0) continue;
      SOUP_CHECK(s.theta && s.grad && s.m && s.v && (state_bits == 32 || (s.m_scale && s.v_scale)),
                 SOUP_ERR_INVALID_ARG, "%s: tensor %d has a null pointer", fn, i);
      SOUP_CHECK(soup_aligned(s.theta, 16) && soup_aligned(s.theta_bf16, 16) && soup_aligned(s.grad, 16) &&
                     soup_aligned(s.m, 16) && soup_aligned(s.v, 16),
                 SOUP_ERR_ALIGN, "%s: tensor %d: theta, theta_bf16, grad, m and v must be 16-byte aligned", fn, i);
      const int64_t v32 = soup_aligned(s.theta, 32) && soup_aligned(s.grad, 32) && soup_aligned(s.m, 32) &&
                          soup_aligned(s.v, 32);
      gt[i] = GroupTensor{s.n, s.theta, s.theta_bf16, s.grad, s.m, s.v, s.m_scale, s.v_scale, v32};
      for (int64_t c = 0; c < chunks_of(s.n); ++c) gc.push_back(GroupChunk{(uint32_t)i, (uint32_t)c});
      total += s.n;
      const size_t gs = grad_type == SOUP_TYPE_F32 ? 4 : 2, ss = state_bits / 8;
      auto add = [&](const void* p, size_t bytes) {
        if (p) ranges.push_back(Range{static_cast<const char*>(p), static_cast<const char*>(p) + bytes, i});
      };
      add(s.theta, s.n * 4);
      add(s.theta_bf16, s.n * 2);
      add(s.grad, s.n * gs);
      add(s.m, s.n * ss);
      add(s.v, s.n * ss);
      if (state_bits == 8) {
        add(s.m_scale, (s.n + 31) / 32);
        add(s.v_scale, (s.n + 31) / 32);
      }
    }
    // every buffer is written by the step: none may share memory with another
    std::sort(ranges.begin(), ranges.end(), [](const Range& x, const Range& y) { return x.lo < y.lo; });
    for (size_t k = 1; k < ranges.size(); ++k)
      SOUP_CHECK(ranges[k].lo >= ranges[k - 1].hi, SOUP_ERR_INVALID_ARG,
                 "%s: buffers of tensors %d and %d overlap", fn, ranges[k - 1].tensor, ranges[k].tensor);
    const size_t need = soup_adamw_group_bytes(tensors, n_tensors);
    SOUP_CHECK(tables_dev && tables_bytes >= need, SOUP_ERR_INVALID_ARG, "%s: %zu bytes of tables, %zu needed", fn,
               tables_bytes, need);
    SOUP_CHECK(soup_aligned(tables_dev, 16), SOUP_ERR_ALIGN, "%s: tables not 16-byte aligned", fn);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(tables_dev);
    const size_t chunks_at = align16(gt.size() * sizeof(GroupTensor));
    SOUP_CUDA_TRY(cudaMemcpyAsync(base, gt.data(), gt.size() * sizeof(GroupTensor), cudaMemcpyHostToDevice, st));
    if (!gc.empty())
      SOUP_CUDA_TRY(
          cudaMemcpyAsync(base + chunks_at, gc.data(), gc.size() * sizeof(GroupChunk), cudaMemcpyHostToDevice, st));
    SOUP_CUDA_TRY(cudaStreamSynchronize(st));
    group->tables = base;
    group->chunks_at = chunks_at;
    group->n_chunks = (int64_t)gc.size();
    group->n_elements = total;
    group->n_tensors = n_tensors;
    group->state_bits = state_bits;
    group->grad_type = grad_type;
  } catch (const std::exception& e) {
    return fail(SOUP_ERR_INVALID_ARG, "%s: host memory: %s", fn, e.what());
  }
  return SOUP_OK;
}

extern "C" soup_status soup_adamw_group_step(const soup_adamw_group* group, float lr, float beta1, float beta2,
                                             float eps, float weight_decay, float grad_scale, int64_t t, uint32_t seed,
                                             int32_t zero_grad, int32_t* nonfinite_dev, void* stream) {
  const char* fn = "soup_adamw_group_step";
  SOUP_CHECK(group && group->tables && group->n_chunks >= 0, SOUP_ERR_INVALID_ARG, "%s: group not initialised", fn);
  SOUP_CHECK((group->state_bits == 8 || group->state_bits == 32) &&
                 (group->grad_type == SOUP_TYPE_F32 || group->grad_type == SOUP_TYPE_BF16),
             SOUP_ERR_INVALID_ARG, "%s: group not initialised", fn);
  SOUP_CHECK(t >= 1, SOUP_ERR_INVALID_ARG, "%s: the step index t starts at 1", fn);
  SOUP_CHECK(beta1 >= 0.f && beta1 < 1.f && beta2 >= 0.f && beta2 < 1.f && eps > 0.f && lr >= 0.f &&
                 weight_decay >= 0.f,
             SOUP_ERR_INVALID_ARG, "%s: need 0 <= beta < 1, eps > 0, lr >= 0, weight_decay >= 0", fn);
  if (group->n_chunks == 0) return SOUP_OK;
  // bias corrections in double on the host
  const double bc1 = 1.0 - std::pow((double)beta1, (double)t);
  const double bc2 = 1.0 - std::pow((double)beta2, (double)t);
  const char* base = static_cast<const char*>(group->tables);
  GroupArgs a;
  a.tensors = reinterpret_cast<const GroupTensor*>(base);
  a.chunks = reinterpret_cast<const GroupChunk*>(base + group->chunks_at);
  a.n_chunks = group->n_chunks;
  a.decay = (float)(1.0 - (double)lr * (double)weight_decay);
  a.beta1 = beta1;
  a.one_minus_beta1 = (float)(1.0 - (double)beta1);
  a.beta2 = beta2;
  a.one_minus_beta2 = (float)(1.0 - (double)beta2);
  a.step_size = (float)((double)lr / bc1);
  a.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(bc2));
  a.eps = eps;
  a.grad_scale = grad_scale;
  a.zero_grad = zero_grad ? 1 : 0;
  a.tiny_eps = eps < 1e-12f * a.inv_sqrt_bc2;
  a.seed = seed;
  a.t = (uint32_t)t;
  a.nonfinite = nonfinite_dev;
  const bool g16 = group->grad_type == SOUP_TYPE_BF16;
  const unsigned grid = (unsigned)std::min<int64_t>(group->n_chunks, (int64_t)sm_count() * 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const double gb = g16 ? 2 : 4;
  profile_begin(st, GC_ADAMW, 0.0,
                (double)group->n_elements * (10.0 + gb * (zero_grad ? 2 : 1) + (group->state_bits == 32 ? 16.0 : 4.125)));
  auto* kern = group->state_bits == 32 ? (g16 ? adamw_group_kernel<32, true> : adamw_group_kernel<32, false>)
                                       : (g16 ? adamw_group_kernel<8, true> : adamw_group_kernel<8, false>);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = dependent_launch(grid, 256, 0, st, attr);
  SOUP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, a));
  SOUP_LAUNCH_CHECK();
  profile_end(st);
  return SOUP_OK;
}

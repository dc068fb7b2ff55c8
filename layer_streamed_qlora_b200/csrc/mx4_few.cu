// y = x W^T over an MXFP4 W for few tokens.
//
// With T tokens a weight of 4.25 bits does 2 T flops: up to a dozen tokens
// the product is bound by reading W once, and the 256-wide tiles of the GEMM
// engine leave most SMs without work.  Here W is the M side of
// mma.sync.m16n8k16 (16 weight rows by 8 tokens): a CTA owns 16 rows and all
// of K, its 8 warps take K in turns of 128, every thread loads one 16-byte
// block of 32 codes per row and turn straight into registers, and the 8
// partial sums meet in shared memory in warp order.  No tile of W passes
// through shared memory, nothing is split across CTAs, and the order of the
// sums does not depend on the launch.
//
// The order of k inside a turn is free as long as both operands agree: of 8
// neighbouring codes of a thread, the first four and then the last four are
// its four k of one instruction, and x is read in the same order.
//
// One token through 6144 x 4096 takes 6.9 us from L2 and 7.6 from HBM, through
// 28672 x 4096 24 us (2.6 TB/s): reading the codes in this pattern alone takes
// 4.1 and 10.4 us.  The rest is the decode, some 36 instructions per 8 codes
// (integer pipe 60 %, issue slots 68 % busy), and an uneven grid: with three
// CTAs per SM, 1792 CTAs are 4.04 rounds of 444, and of the 384 of 6144 rows
// some SMs get three and some two.  A table of byte pairs in shared memory
// halves the instructions and gained nothing (8.3 and 29 us: its loads compete
// with x's).
#include <algorithm>

#include "linear.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace soup {
namespace {

constexpr int WARPS = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Loads of W and x are ordinary ones: see dependent_launch.
// NT: groups of 8 tokens; DEPTH: turns whose loads of W are in flight together.
template <int NT, int DEPTH>
__global__ void __launch_bounds__(32 * WARPS, NT == 1 ? 3 : 2)
    mx4_few_kernel(const uint8_t* codes, const uint8_t* scales, int N, int K, int64_t scale_stride, const uint16_t* x,
                   int64_t ldx, int T, uint16_t* y, int64_t ldy) {
  __shared__ float part[WARPS][NT * 8][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int row0 = blockIdx.x * 16, blocks = K / 32, turns = (blocks + 3) / 4;
  // No grid_dep_launch: CTAs of the next product that come early take the
  // slots unevenly (4096 x 14336: 15.4 us without, 19.7 with).
  ptx::grid_dep_wait();
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;

  for (int turn0 = warp; turn0 < turns; turn0 += WARPS * DEPTH) {
    uint4 w[DEPTH][2];
    uint32_t s[DEPTH][2];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int b = (turn0 + d * WARPS) * 4 + tq;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row0 + 8 * r + g;
        const bool ok = b < blocks;
        w[d][r] = ok ? reinterpret_cast<const uint4*>(codes + (int64_t)row * (K / 2))[b] : make_uint4(0, 0, 0, 0);
        s[d][r] = ok ? scales[row * scale_stride + b] : 0u;
      }
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int b = (turn0 + d * WARPS) * 4 + tq;
      if (turn0 + d * WARPS >= turns) break;
      uint32_t sc[2];
      bool large = false;  // rare: a scale above 2
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sc[r] = mx4_scale_bf16x2(s[d][r]);
        large |= mx4_is_large(s[d][r]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t bx[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int t = 8 * j + g;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (t < T && b < blocks) v = reinterpret_cast<const uint4*>(x + t * ldx + (int64_t)b * 32)[u];
          bx[j][0] = v.x;
          bx[j][1] = v.y;
          bx[j][2] = v.z;
          bx[j][3] = v.w;
        }
        const uint4 lo = w[d][0], hi = w[d][1];
        uint32_t p[4], q[4];
        mx4_decode8_scaled(u == 0 ? lo.x : u == 1 ? lo.y : u == 2 ? lo.z : lo.w, sc[0], p);
        mx4_decode8_scaled(u == 0 ? hi.x : u == 1 ? hi.y : u == 2 ? hi.z : hi.w, sc[1], q);
        if (large) {
          const uint32_t more[2] = {mx4_is_large(s[d][0]) ? mx4_large_bf16x2(s[d][0]) : 0x3F803F80u,
                                    mx4_is_large(s[d][1]) ? mx4_large_bf16x2(s[d][1]) : 0x3F803F80u};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            p[k] = mul_bf16x2(p[k], more[0]);
            q[k] = mul_bf16x2(q[k], more[1]);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma16816(acc[j], p[0], q[0], p[1], q[1], bx[j][0], bx[j][1]);
          mma16816(acc[j], p[2], q[2], p[3], q[3], bx[j][2], bx[j][3]);
        }
      }
    }
  }
  // acc[j]: rows g (+ 8), tokens 8 j + 2 tq (+ 1)
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) part[warp][8 * j + 2 * tq + (k & 1)][g + 8 * (k >> 1)] = acc[j][k];
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * NT * 8; e += 32 * WARPS) {
    const int r = e % 16, t = e / 16;
    if (t >= T) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += part[k][t][r];
    const __nv_bfloat16 o = __float2bfloat16_rn(v);
    y[t * ldy + row0 + r] = *reinterpret_cast<const uint16_t*>(&o);
  }
}

template <int NT, int DEPTH>
soup_status launch_few(const soup_weight* W, const uint16_t* x, int64_t ldx, int T, uint16_t* y, int64_t ldy,
                       cudaStream_t st) {
  const int N = (int)W->out_features, K = (int)W->in_features;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = dependent_launch(N / 16, 32 * WARPS, 0, st, attr);
  SOUP_CUDA_TRY(cudaLaunchKernelEx(&cfg, mx4_few_kernel<NT, DEPTH>, W->codes, W->scales, N, K, mx4_scale_stride(K), x,
                                   ldx, T, y, ldy));
  SOUP_LAUNCH_CHECK();
  return SOUP_OK;
}

}  // namespace

soup_status mx4_few(const soup_weight* W, const uint16_t* x, int64_t ldx, int T, uint16_t* y, int64_t ldy,
                    cudaStream_t st) {
  const double n = (double)W->out_features * W->in_features;
  profile_begin(st, GC_NF4_FWD, 2.0 * T * n, n * (0.5 + 1.0 / 32) + 2.0 * T * (W->out_features + W->in_features));
  soup_status r;
  if (T <= 8) r = launch_few<1, 4>(W, x, ldx, T, y, ldy, st);
  else r = launch_few<2, 2>(W, x, ldx, T, y, ldy, st);
  SOUP_TRY(r);
  profile_end(st);
  return SOUP_OK;
}

}  // namespace soup

// The frozen MXFP4 product for some dozens to some hundreds of tokens, on
// tcgen05 with the weights as the M side: D[128 weight rows, tokens] per CTA,
//   forward   y^T = W x^T     A = W rows, K-major            (K = in)
//   backward  dx^T = W^T dy^T A = W columns, MN-major        (K = out)
//
// The GEMM engine's tiles have 256 tokens by 256 weight rows per CTA pair:
// with few tokens most of a tile is padding, and a projection has too few
// tiles for the GPU.  With the tokens as N the tile is as wide as T needs (16
// to 256 columns), and K is cut over a cluster of up to 4 CTAs, so that
// tiles times slices is about the number of SMs.  The slices' sums meet in
// distributed shared memory: every CTA leaves its fp32 partial in its own
// shared memory and finishes a share of the tokens, adding the partials in
// slice order (the same bits on every run, no workspace, no second launch).
//
// Warps: 0 TMA of the x tiles, 1 MMA, 2 TMA of codes and scales, 3..18 decode:
// four groups of 4, one for each of the four k-blocks of a code load; a thread
// turns two blocks of 32 codes into bf16 (two, to share the waits, fences and
// addresses).  In the forward a thread's 64 values are one row of A, and go to
// tensor memory as the A operand: neither the stores nor the MMA's reads of A
// take shared memory's port then (256 tokens through 28672 x 4096: 65 -> 57
// us when it was changed, 55 now).  In the backward they are parts of 64 rows, and go to the swizzled
// stage in shared memory.
//
// What bounds it (forward, one CTA per SM, cycles per k-block from the slope
// over K): 490 with up to 64 tokens, 620 with 176, 730 with 256.  With the
// decode left out 300 remain of the 490, and all of the 730: there the x tile
// is the limit, 32 KB per k-block and SM from L2 (45 bytes a clock), and the
// tensor core needs 512.  Weights in L2 instead of HBM make no difference.
// The slice count (1, 2 or 4) leaves SMs idle beside that: 48 row tiles (6144
// rows) run on 96 of 148, 112 tiles on 112, and 224 take two rounds for 1.5.
// 256 tokens through 28672 x 4096 take 55 us (1090 TFLOP/s), 64 take 44 us; the
// GEMM engine's 256-token tiles take 62 us for either.  The start of a launch
// (barriers, tensor memory) runs while the kernel before it ends: calls of 77
// tokens backward through 2560 x 2016 14.0 -> 10.6 us apart, 7 of which the
// host takes for a call.

#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "linear.h"
#include "mx4.cuh"
#include "ptx.cuh"

namespace soup {
namespace {

constexpr int ROWS = 128;             // weight rows (columns) per CTA
constexpr int A_BYTES = ROWS * 128;   // one 64-wide k-block of A
constexpr int MAX_STAGES = 8;  // of the A ring and of the x ring
// Decode groups, and warps of one.
constexpr int GROUPS = 4, GROUP_WARPS = 4;
// Codes come CODE_KB k-blocks at a time, one for each group: 128 rows x 128
// bytes (swizzled) and 16 scale bytes per row (of 8 k-blocks, two loads'
// worth), or 256 k-rows x 64 bytes and 16 scale bytes per k-row.
constexpr int CODE_KB = GROUPS, CODE_SLOTS = 3;
template <bool TRANS>
struct Codes {
  static constexpr int BYTES = 16384, SCALE_BYTES = TRANS ? 4096 : 2048;
  static constexpr int ALL = CODE_SLOTS * (BYTES + SCALE_BYTES);
};
// A decode group that waits for the stage of k-block i has waited for the one
// of k-block i - CODE_KB before.  The wait's parity tells this phase from the
// one before only if that one is over: i - CODE_KB - stages >= i - 2 stages.
constexpr int MIN_A_STAGES = CODE_KB;
// Tensor memory of the forward: the accumulator's columns, then MAX_STAGES
// stages of A with 32 columns each.
constexpr uint32_t A_COL = 256;
constexpr int THREADS = 32 * (3 + GROUP_WARPS * GROUPS);
constexpr int BAR_BYTES = 512;

struct MidArgs {
  int M, K, T;        // M: outputs per token; K: summed
  int bn;             // tokens per tile, a multiple of 16
  int a_stages, x_stages, slices;
  uint16_t* y;
  int64_t ldy;
  int* err;
  long long wait_limit;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t* v) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// Two blocks of 32 codes with the two bytes of scales, of which the first
// `left` are in the matrix and the others are zeros.
__device__ __forceinline__ void decode_64(uint32_t* w, uint32_t sc, int left, uint32_t* v) {
  if (left < 2) {
    w[4] = w[5] = w[6] = w[7] = 0;
    sc &= 0xFF;
    if (left < 1) w[0] = w[1] = w[2] = w[3] = sc = 0;
  }
  mx4_decode<4>(w, sc & 0xFF, v);
  mx4_decode<4>(w + 4, sc >> 8, v + 16);
}

// By one lane of a warp, and by all lanes with one answer.
#define MID_FAILED (atomicOr(a.err, 1), *abort_flag = 1, false)
#define MID_WAIT_LANE(bar, parity) (ptx::mbar_wait_bounded((bar), (parity), abort_flag, a.wait_limit) || MID_FAILED)
#define MID_WAIT(bar, parity) (ptx::mbar_wait_warp((bar), (parity), abort_flag, a.wait_limit) || MID_FAILED)

template <bool TRANS>
__global__ void __launch_bounds__(THREADS) mx4_mid_kernel(const __grid_constant__ CUtensorMap tmx,
                                                          const __grid_constant__ CUtensorMap tmc,
                                                          const __grid_constant__ CUtensorMap tms, const MidArgs a) {
  using CO = Codes<TRANS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int b_bytes = a.bn * 128, a_stages = a.a_stages, x_stages = a.x_stages;
  const int a_ring = TRANS ? a_stages * A_BYTES : 0;  // forward: in tensor memory
  uint8_t* sA = sm;
  uint8_t* sB = sA + a_ring;
  uint8_t* sC = sB + x_stages * b_bytes;
  uint8_t* sS = sC + CODE_SLOTS * CO::BYTES;
  // the partial sums [bn][ROWS] fp32 take the stages' place when K is done
  const int ring = a_ring + x_stages * b_bytes + CO::ALL, parts = a.bn * ROWS * 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + (ring > parts ? ring : parts));
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* xfull = empty + MAX_STAGES;
  uint64_t* xempty = xfull + MAX_STAGES;
  uint64_t* cfull = xempty + MAX_STAGES;
  uint64_t* cempty = cfull + CODE_SLOTS;
  uint64_t* accf = cempty + CODE_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // warp-uniform, and known to the compiler as such (see the TMA and MMA loops)
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int slice = (int)blockIdx.x % a.slices, m0 = (int)blockIdx.x / a.slices * ROWS, t0 = (int)blockIdx.y * a.bn;
  const int num_kb = (a.K + 63) / 64;
  // slices of whole code loads
  const int loads = (num_kb + CODE_KB - 1) / CODE_KB;
  const int kb0 = (int)((int64_t)slice * loads / a.slices) * CODE_KB;
  const int kb1 = min((int)((int64_t)(slice + 1) * loads / a.slices) * CODE_KB, num_kb);
  const int nk = kb1 - kb0;
  const uint32_t cols = !TRANS ? 512 : (a.bn <= 32 ? 32 : (a.bn <= 64 ? 64 : (a.bn <= 128 ? 128 : 256)));

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      ptx::mbar_init(&full[s], GROUP_WARPS);
      ptx::mbar_init(&empty[s], 1);
      ptx::mbar_init(&xfull[s], 1);
      ptx::mbar_init(&xempty[s], 1);
    }
    for (int g = 0; g < CODE_SLOTS; ++g) {
      ptx::mbar_init(&cfull[g], 1);
      ptx::mbar_init(&cempty[g], GROUP_WARPS * GROUPS);
    }
    ptx::mbar_init(accf, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmc);
    ptx::prefetch_tmap(&tms);
    ptx::prefetch_tmap(&tmx);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::grid_dep_wait();
  ptx::grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);

  if (warp == 0) {
    if (ptx::elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < nk; ++i) {
        if (!MID_WAIT_LANE(&xempty[s], ph ^ 1)) break;
        ptx::mbar_arrive_expect_tx(&xfull[s], (uint32_t)b_bytes);
        ptx::tma_load_2d(sB + s * b_bytes, &tmx, &xfull[s], (kb0 + i) * 64, t0);
        if (++s == x_stages) { s = 0; ph ^= 1; }
      }
    }
  } else if (warp == 2) {
    if (ptx::elect_one()) {
      int g = 0;
      uint32_t gph = 0;
      for (int kb = kb0; kb < kb1; kb += CODE_KB) {
        if (!MID_WAIT_LANE(&cempty[g], gph ^ 1)) break;
        ptx::mbar_arrive_expect_tx(&cfull[g], CO::BYTES + CO::SCALE_BYTES);
        ptx::tma_load_2d(sC + g * CO::BYTES, &tmc, &cfull[g], TRANS ? m0 / 2 : kb * 32, TRANS ? kb * 64 : m0);
        ptx::tma_load_2d(sS + g * CO::SCALE_BYTES, &tms, &cfull[g], (TRANS ? m0 / 32 : kb * 2) & ~15,
                         TRANS ? kb * 64 : m0);
        if (++g == CODE_SLOTS) { g = 0; gph ^= 1; }
      }
    }
  } else if (warp == 1) {
    // descriptors are advanced, not built
    if (ptx::elect_one()) {
      const uint32_t idesc = ptx::idesc_bf16(ROWS, a.bn, TRANS ? 1 : 0, 0);
      constexpr uint32_t HI = ptx::desc_hi_sw128(1024);
      constexpr uint32_t A_STEP = TRANS ? 2048 >> 4 : 2;
      const uint32_t a0 = ptx::desc_lo(ptx::smem_u32(sA), TRANS ? 8192 : 16);
      const uint32_t b0 = ptx::desc_lo(ptx::smem_u32(sB), 16);
      int s = 0, xs = 0;
      uint32_t ph = 0, xph = 0;
      bool ok = true, ready = false;
      for (int i = 0; i < nk; ++i) {
        if (!ready && (!MID_WAIT_LANE(&xfull[xs], xph) || !MID_WAIT_LANE(&full[s], ph))) { ok = false; break; }
        const uint32_t alo = a0 + s * (A_BYTES >> 4), blo = b0 + xs * (b_bytes >> 4), ta = tmem + A_COL + s * 32;
        ptx::tc_fence_after();
        uint64_t *const done = &empty[s], *const xdone = &xempty[xs];
        if (++s == a_stages) { s = 0; ph ^= 1; }
        if (++xs == x_stages) { xs = 0; xph ^= 1; }
        // the next k-block's barriers are tried before this one's MMAs are
        // issued: a try takes 60 cycles to answer
        const bool r0 = ptx::mbar_try_wait(&xfull[xs], xph), r1 = ptx::mbar_try_wait(&full[s], ph);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t bd = ptx::desc_of(blo + k * 2, HI);
          const uint32_t acc = (i > 0 || k > 0) ? 1u : 0u;
          if (TRANS) ptx::mma_bf16(tmem, ptx::desc_of(alo + k * A_STEP, HI), bd, idesc, acc);
          else ptx::mma_bf16_ta(tmem, ta + k * 8, bd, idesc, acc);
        }
        ptx::mma_commit(done);
        ptx::mma_commit(xdone);
        ready = r0 && r1;
      }
      if (ok) ptx::mma_commit(accf);
    }
  } else {
    // forward: weight row t, its 64 codes of the group's k-block; backward:
    // k-row t / 2 of it, 64 of the 128 columns
    const int group = (warp - 3) / GROUP_WARPS, q = warp & 3, t = TRANS ? (threadIdx.x - 96) & 127 : q * 32 + lane;
    const int r = TRANS ? t >> 1 : t, h = TRANS ? t & 1 : 0;
    // its two 16-byte units of codes (128-byte swizzled rows in the forward)
    const uint32_t c0 = ptx::smem_u32(sC) + (TRANS ? group * 4096 + r * 64 + h * 32 : r * 128 + (((group * 2) ^ (r & 7)) << 4));
    const uint32_t c1 = c0 ^ 16;
    // its two scale bytes: a window of 16 holds 8 k-blocks, two code loads' worth
    const uint32_t s0 = ptx::smem_u32(sS) + (TRANS ? (group * 64 + r) * 16 + (m0 / 32 & 15) + h * 2 : r * 16 + group * 2);
    // TMA reads zeros beyond the matrix, but a row can end inside its padded
    // scales: blocks from `blocks` on are none
    const int blocks = TRANS ? (a.M - m0 - h * 64 + 31) / 32 : (m0 + r < a.M ? a.K / 32 : 0);
    // where its 64 values go: tensor memory, or a row of the swizzled stage
    const uint32_t dst = TRANS ? ptx::smem_u32(sA + h * 8192 + r * 128) ^ ((r & 7) << 4)
                               : tmem + ((uint32_t)(q * 32) << 16) + A_COL;
    int s = group, g = 0;
    uint32_t ph = 0, gph = 0;
    for (int kb = kb0; kb + group < kb1; kb += CODE_KB) {
      if (!MID_WAIT(&cfull[g], gph)) break;
      uint32_t w[8], v[32];
      ld_shared_v4(c0 + g * CO::BYTES, w);
      ld_shared_v4(c1 + g * CO::BYTES, w + 4);
      const uint32_t sc = ld_shared_u16(s0 + g * CO::SCALE_BYTES + (TRANS ? 0 : (kb & 4) * 2));
      const bool free_now = __all_sync(0xFFFFFFFFu, ptx::mbar_try_wait(&empty[s], ph ^ 1));
      decode_64(w, sc, TRANS ? blocks : blocks - (kb + group) * 2, v);
      if (!free_now && !MID_WAIT(&empty[s], ph ^ 1)) break;
      if (TRANS) {
        const uint32_t o = dst + s * A_BYTES;
#pragma unroll
        for (int u = 0; u < 8; ++u) st_shared_v4(o ^ (u << 4), v + 4 * u);
        ptx::fence_proxy_async_smem();
      } else {
        ptx::tc_fence_after();
        ptx::tmem_st32(dst + s * 32, v);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&full[s]);
        ptx::mbar_arrive(&cempty[g]);
      }
      if (++g == CODE_SLOTS) { g = 0; gph ^= 1; }
      s += GROUPS;
      if (s >= a_stages) { s -= a_stages; ph ^= 1; }
    }
    // the accumulator to shared memory as [token][row]: the stages are free
    // once every MMA has completed
    if (MID_WAIT(accf, 0)) {
      ptx::tc_fence_after();
      float* part = reinterpret_cast<float*>(sm) + q * 32 + lane;
      for (int c = (warp - 3) >> 2; c < a.bn / 16; c += GROUPS) {
        uint32_t v[16];
        ptx::tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c * 16, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) part[(c * 16 + k) * ROWS] = __uint_as_float(v[k]);
      }
    }
    ptx::tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag) {
    // let copies and MMAs already in flight land (bounded: about 1 ms)
    const long long c0 = clock64();
    while (clock64() - c0 < 2000000LL) {
    }
  }
  if (a.slices > 1) ptx::cluster_sync();
  if (!*abort_flag) {
    // this CTA's share of the tile's tokens: the slices' partials in order
    const int per = (a.bn + a.slices - 1) / a.slices;
    const uint32_t base = ptx::smem_u32(sm) + lane * 16;
    const int m = m0 + lane * 4;
    for (int t = slice * per + warp; t < min((slice + 1) * per, a.bn); t += THREADS / 32) {
      if (t0 + t >= a.T) break;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int p = 0; p < a.slices; ++p) {
        const uint32_t at = base + t * ROWS * 4;
        const float4 x = ld_cluster_f4(a.slices > 1 ? ptx::mapa_shared(at, p) : at);
        v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
      }
      if (m < a.M) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(a.y + (int64_t)(t0 + t) * a.ldy + m) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
  if (a.slices > 1) ptx::cluster_sync();  // no CTA leaves while another reads its partial
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, cols);
  }
}

constexpr int CU_U8 = 0, CU_BF16 = 9;  // CU_TENSOR_MAP_DATA_TYPE_*
constexpr int CU_SWIZZLE_128 = 3;

soup_status make_map(CUtensorMap* m, const void* p, int type, int64_t cols, int64_t rows, int64_t row_bytes,
                     uint32_t box_cols, uint32_t box_rows, int swizzle, const char* what) {
  EncodeTiledFn enc = encode_tiled();
  SOUP_CHECK(enc != nullptr, SOUP_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const uint64_t gdim[2] = {(uint64_t)cols, (uint64_t)rows}, gstride[1] = {(uint64_t)row_bytes};
  const uint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
  const int r = enc(m, type, 2, const_cast<void*>(p), gdim, gstride, box, estr, 0, swizzle, 3 /* L2 promotion 256 B */, 0);
  SOUP_CHECK(r == 0, SOUP_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with %d", what, r);
  return SOUP_OK;
}

template <bool TRANS>
soup_status launch_mid(const CUtensorMap (&map)[3], const MidArgs& a, dim3 grid, size_t smem, cudaStream_t st) {
  auto kern = mx4_mid_kernel<TRANS>;
  SOUP_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448));
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = dependent_launch(grid, THREADS, smem, st, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.slices;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  SOUP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kern, map[0], map[1], map[2], a));
  SOUP_LAUNCH_CHECK();
  return SOUP_OK;
}

}  // namespace

soup_status mx4_mid(const soup_weight* W, bool trans, const uint16_t* x, int64_t ldx, int T, uint16_t* y, int64_t ldy,
                    cudaStream_t st) {
  MidArgs a;
  memset(&a, 0, sizeof(a));
  a.M = (int)(trans ? W->in_features : W->out_features);
  a.K = (int)(trans ? W->out_features : W->in_features);
  a.T = T;
  a.y = y;
  a.ldy = ldy;
  const int ttiles = (T + 255) / 256;
  a.bn = ((T + ttiles - 1) / ttiles + 15) / 16 * 16;
  const int rtiles = (a.M + ROWS - 1) / ROWS, num_kb = (a.K + 63) / 64;
  // up to 4 slices: clusters of 8 one-per-SM CTAs do not find room at once
  // (64 tokens through 2048 x 11008: 30 us with 8 slices, 21.5 with 4, 33 with 2)
  a.slices = 1;
  while (a.slices < 4 && rtiles * ttiles * a.slices * 2 <= sm_count() && num_kb / (a.slices * 2) >= GROUPS) a.slices *= 2;
  a.err = device_error_word();
  SOUP_CHECK(a.err != nullptr, SOUP_ERR_CUDA, "device error word unavailable");
  a.wait_limit = 4000000000LL;
  const int codes = trans ? Codes<true>::ALL : Codes<false>::ALL, room = 232448 - 1024 - BAR_BYTES - codes;
  const int xb = a.bn * 128;
  a.x_stages = std::min(MAX_STAGES, (room - (trans ? MIN_A_STAGES * A_BYTES : 0)) / xb);  // 3 (5) at bn = 256
  a.a_stages = trans ? std::min(MAX_STAGES, (room - a.x_stages * xb) / A_BYTES) : MAX_STAGES;
  SOUP_CHECK(a.x_stages >= 2 && a.a_stages >= MIN_A_STAGES, SOUP_ERR_SHAPE, "frozen linear: %d tokens per tile", a.bn);
  // at least half of an SM's shared memory: a CTA that holds tensor memory and
  // waits for its cluster must not share an SM with one that waits for the rest
  const size_t smem = std::max<size_t>(
      1024 + std::max((trans ? a.a_stages * A_BYTES : 0) + a.x_stages * xb + codes, a.bn * ROWS * 4) + BAR_BYTES, 120 << 10);
  CUtensorMap map[3];
  const int64_t out = W->out_features, in = W->in_features;
  SOUP_TRY(make_map(&map[0], x, CU_BF16, a.K, T, ldx * 2, 64, (uint32_t)a.bn, CU_SWIZZLE_128, "x"));
  SOUP_TRY(make_map(&map[1], W->codes, CU_U8, in / 2, out, in / 2, trans ? 64 : 128, trans ? 256 : 128,
                    trans ? 0 : CU_SWIZZLE_128, "codes"));
  SOUP_TRY(make_map(&map[2], W->scales, CU_U8, mx4_scale_stride(in), out, mx4_scale_stride(in), 16,
                    trans ? 256 : 128, 0, "scales"));
  const double n = (double)W->out_features * W->in_features;
  profile_begin(st, trans ? GC_NF4_BWD : GC_NF4_FWD, 2.0 * T * n,
                n * (0.5 + 1.0 / 32) + 2.0 * T * (W->out_features + W->in_features));
  const dim3 grid(rtiles * a.slices, ttiles);
  if (trans) SOUP_TRY(launch_mid<true>(map, a, grid, smem, st));
  else SOUP_TRY(launch_mid<false>(map, a, grid, smem, st));
  profile_end(st);
  return SOUP_OK;
}

}  // namespace soup

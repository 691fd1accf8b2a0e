// E4M3 quantisation of rows with one fp32 scale for each block of 128 columns:
//
//   s = fp32(max|v|) / 448,  q = e4m3_rne_saturate(v / s)   (IEEE fp32 division)
//   an all-zero block gets s = 1 and q = 0
//
// the rule of quant.hip with a block in a row's place.  Codes and scales lie row
// by row, so a matrix is one run of blocks.  Sixteen lanes hold a block, eight
// consecutive elements each.
//
// SwiGLU form: v = silu(g) * u in fp32 from two matrices of 32-bit sums.
#include "e4m3.h"
#include "kernels.h"

namespace moe {

constexpr int kQbThreads = 256;
constexpr int kQbLanes = 16;                       // lanes to a block
constexpr int kQbBlocks = kQbThreads / kQbLanes;  // blocks of a workgroup at a time

enum : int { kQbBf16 = 0, kQbF32 = 1, kQbSwiglu = 2 };

// amax / 448 of a block.  fp32 rows may be so small that the quotient rounds to
// zero: the smallest number then, so that codes stand for multiples of something.
__device__ __forceinline__ float qb_scale(float amax) {
  return amax == 0.0f ? 1.0f : fmaxf(amax / 448.0f, __uint_as_float(1u));
}

template <int KIND>
__global__ __launch_bounds__(kQbThreads) void quant_blocks_kernel(const void *__restrict__ x,
                                                                  const void *__restrict__ x2,
                                                                  long long blocks,
                                                                  uint8_t *__restrict__ q,
                                                                  float *__restrict__ s) {
  const int sub = threadIdx.x & (kQbLanes - 1);
  const long long step = (long long)gridDim.x * kQbBlocks;
  // whole waves: a wave's blocks end together or past the end
  for (long long b = (long long)blockIdx.x * kQbBlocks + threadIdx.x / kQbLanes;; b += step) {
    if (!__any(b < blocks)) break;
    const bool on = b < blocks;
    const size_t at = (size_t)(on ? b : blocks - 1) * 128 + sub * 8;
    float v[8];
    if constexpr (KIND == kQbBf16) {
      const i32x4 raw = *reinterpret_cast<const i32x4 *>(static_cast<const uint16_t *>(x) + at);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[2 * w] = __uint_as_float((uint32_t)raw[w] << 16);
        v[2 * w + 1] = __uint_as_float((uint32_t)raw[w] & 0xffff0000u);
      }
    } else {
      const f32x4 *p = reinterpret_cast<const f32x4 *>(static_cast<const float *>(x) + at);
      const f32x4 lo = p[0], hi = p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = lo[e];
        v[4 + e] = hi[e];
      }
      if constexpr (KIND == kQbSwiglu) {
        const f32x4 *p2 = reinterpret_cast<const f32x4 *>(static_cast<const float *>(x2) + at);
        const f32x4 ulo = p2[0], uhi = p2[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = swiglu(v[e], ulo[e]);
          v[4 + e] = swiglu(v[4 + e], uhi[e]);
        }
      }
    }
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
#pragma unroll
    for (int m = kQbLanes / 2; m > 0; m >>= 1) amax = fmaxf(amax, __shfl_xor(amax, m));
    const bool zero = amax == 0.0f;
    const float sc = qb_scale(amax);
    bool exact;
    const float rcp = quant_rcp(sc, &exact);
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    uint2 out;
    out.x = quant_e4m3_x4(lo, sc, rcp, exact, zero);
    out.y = quant_e4m3_x4(hi, sc, rcp, exact, zero);
    if (on) {
      *reinterpret_cast<uint2 *>(q + at) = out;
      if (sub == 0) s[b] = sc;
    }
  }
}

static int qb_grid(long long blocks, int grid_cap) {
  const long long want = (blocks + kQbBlocks - 1) / kQbBlocks;
  const long long cap = (long long)grid_cap * 4;
  return (int)(want < cap ? want : cap);
}

hipError_t launch_quant_blocks(const void *x, bool f32, long long blocks, uint8_t *q, float *s,
                               int grid_cap, hipStream_t stream) {
  const dim3 grid(qb_grid(blocks, grid_cap)), block(kQbThreads);
  if (f32)
    return launch(quant_blocks_kernel<kQbF32>, grid, block, stream, x, nullptr, blocks, q, s);
  return launch(quant_blocks_kernel<kQbBf16>, grid, block, stream, x, nullptr, blocks, q, s);
}

hipError_t launch_quant_swiglu(const float *g, const float *u, long long blocks, uint8_t *q,
                               float *s, int grid_cap, hipStream_t stream) {
  return launch(quant_blocks_kernel<kQbSwiglu>, dim3(qb_grid(blocks, grid_cap)), dim3(kQbThreads),
                stream, g, u, blocks, q, s);
}

}  // namespace moe

// E4M3 quantisation of rows with one fp32 scale for each block of 128 columns:
//
//   s = fp32(max|v|) / 448,  q = e4m3_rne_saturate(v / s)   (IEEE fp32 division)
//   an all-zero block gets s = 1 and q = 0
//
// the rule of quant.hip with a block in a row's place.  Codes and scales lie row
// by row, so a matrix is one run of blocks.  Sixteen lanes hold a block, eight
// consecutive elements each.
//
// Bound by memory: 8192 rows of 4096 take 17.5 us on MI355X in bf16 (5.8 TB/s over what
// is read and written, where a large copy reaches 5.2) and 29.5 in fp32 (5.7), calls one
// after another on inputs in turn.  It took 32 in bf16 as long as quotients near a midpoint of two codes, which bf16 numbers have
// often, were divided behind a branch (quant_e4m3_x4); four fused multiply-adds give
// every quotient correctly rounded (qb_div).  Two or four blocks to a lane at a time:
// nothing at this size, 0.2 to 0.8 us slower for 401 rows.  Codes stored past the
// caches: nothing, and the product that reads them 2 to 4% slower.
#include "e4m3.h"
#include "kernels.h"

namespace moe {

constexpr int kQbThreads = 256;
constexpr int kQbBlocks = kQbThreads / kQbLanes;  // blocks of a workgroup at a time

template <int KIND>
__global__ __launch_bounds__(kQbThreads) void quant_blocks_kernel(const void *__restrict__ x,
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
    float v[8], sc;
    qb_load<KIND>(x, at, v);
    const uint2 out = qb_codes(v, &sc);
    if (on) {
      *reinterpret_cast<uint2 *>(q + at) = out;
      if (sub == 0) s[b] = sc;
    }
  }
}

hipError_t launch_quant_blocks(const void *x, bool f32, long long blocks, uint8_t *q, float *s,
                               hipStream_t stream) {
  // sixteen workgroups to each of 256 compute units at the most, each looping over blocks
  const long long want = (blocks + kQbBlocks - 1) / kQbBlocks;
  const dim3 grid((unsigned)(want < 4096 ? want : 4096)), block(kQbThreads);
  if (f32) return launch(quant_blocks_kernel<kQbF32>, grid, block, stream, x, blocks, q, s);
  return launch(quant_blocks_kernel<kQbBf16>, grid, block, stream, x, blocks, q, s);
}

}  // namespace moe

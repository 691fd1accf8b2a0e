// The 8-bit product of matmul_fp8.hip for few rows, where it is a stream of weights:
//
//   y[m, n] = sum over blocks b of 128 columns of
//             (xs[m, b] * ws[n / 128, b]) * sum over c in b of x[m, c] * w[n, c]
//
// A workgroup takes 16 weight rows (of the gate/up form 8 rows of each matrix) and
// all columns; its waves take the blocks of columns in turn and add up their sums
// in LDS at the end, in the order of the waves.  A wave loads a block's weights
// straight into registers, 16 rows of 128 bytes, and multiplies them with up to
// 16 rows of x.  Codes go through the 16x16x32 bf16 instruction as bf16
// numbers, which hold them: the products are exact and the sums fp32's (the 8-bit
// instructions drop bits, matmul_fp8.hip), and the matrix unit has nothing else to do.
//
// Few elements of x that come in bf16 or fp32 are quantised by every workgroup for
// itself, into LDS, while its first weights are under way: 16 elements to a thread
// at most (MI355X, 4096 x 4096: one row 0.7 us, where a launch of its own takes 2.2).
//
// Bound by the weights' stream and its start: one row by 4096 x 4096 5.0 us in a graph,
// 5.8 in a trace, of which an empty launch is 2.2 and 16.8 MB at 6.2 TB/s 2.7.
#include "e4m3.h"
#include "kernels.h"

namespace moe {

constexpr int kMvWaves = 8;
constexpr int kMvThreads = kMvWaves * kWave;
constexpr int kMvAhead = 4;  // blocks of a wave that are loaded together
// Elements of x that a workgroup quantises, eight to a thread at a time.
constexpr int kMvPasses = 2;
constexpr int kMvQuant = kMvPasses * kMvThreads * 8;
static_assert(kMvQuant == kMatvecQuant, "what the rule takes for granted");
static_assert((long long)kMatvecCols / 8 * kMvThreads < 1LL << 32, "one line of workgroups");
constexpr int kMvPad = 16;  // bytes behind a row of codes: rows start in different banks

enum : int { kMvCodes = 2 };  // beside kQbBf16 and kQbF32

template <int KIND, bool GATEUP>
__global__ __launch_bounds__(kMvThreads) void matvec_fp8_kernel(MatvecArgs a) {
  constexpr int FEAT = GATEUP ? 8 : 16;  // columns of y
  constexpr int kSums = kMvWaves * 256 * 4;
  constexpr bool QUANT = KIND != kMvCodes;
  constexpr int kCodes = kMvQuant + 16 * kMvPad + kMvQuant / 128 * 4;
  constexpr int kRoom = QUANT && kCodes > kSums ? kCodes : kSums;
  __shared__ __attribute__((aligned(16))) uint8_t room[kRoom];
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int row = lane & 15, quarter = lane >> 4;
  const int K = a.K, KB = K / 128;
  const int n0 = blockIdx.x * FEAT;  // of at most kMatvecCols

  // this lane's weight row, and the scales of the rows that its sums belong to
  const uint8_t *w;
  const float *ws;
  if (GATEUP) {
    w = (row < 8 ? a.w0 : a.w1) + (size_t)(n0 + (row & 7)) * K;
    ws = (quarter < 2 ? a.s0 : a.s1) + (size_t)(n0 / 128) * KB;
  } else {
    w = a.w0 + (size_t)(n0 + min(row, a.N - 1 - n0)) * K;
    ws = a.s0 + (size_t)(n0 / 128) * KB;
  }
  w += quarter * 16;
  // chunks of block b: bytes [16 quarter, +16) and those 64 further on
  i32x4 wr[kMvAhead][2];
  float wsc[kMvAhead];
  auto load = [&](int first) {
#pragma unroll
    for (int i = 0; i < kMvAhead; ++i) {
      const int b = min(first + i * kMvWaves, KB - 1);
      const i32x4 *p = reinterpret_cast<const i32x4 *>(w + (size_t)b * 128);
      wr[i][0] = __builtin_nontemporal_load(p);
      wr[i][1] = __builtin_nontemporal_load(p + 4);
      wsc[i] = ws[b];
    }
  };
  // The elements to quantise are loaded ahead of the weights: loads come back in order.
  const int sub = threadIdx.x & (kQbLanes - 1), total = a.M * KB;
  float v[kMvPasses][8];
  if constexpr (QUANT) {
#pragma unroll
    for (int i = 0; i < kMvPasses; ++i) {
      const int at = min((int)threadIdx.x / kQbLanes + i * (kMvThreads / kQbLanes), total - 1);
      qb_load<KIND>(a.x, (size_t)at * 128 + sub * 8, v[i]);
    }
  }
  load(wv);

  const int stride = K + kMvPad;
  float *const scales = reinterpret_cast<float *>(room + (size_t)a.M * stride);
  if constexpr (QUANT) {
#pragma unroll
    for (int i = 0; i < kMvPasses; ++i) {
      const int at = threadIdx.x / kQbLanes + i * (kMvThreads / kQbLanes);
      if (!__any(at < total)) break;
      float sc;
      const uint2 codes = qb_codes(v[i], &sc);
      if (at < total) {
        const int m = at / KB, b = at - m * KB;
        *reinterpret_cast<uint2 *>(room + m * stride + b * 128 + sub * 8) = codes;
        if (sub == 0) scales[at] = sc;
      }
    }
    __syncthreads();
  }

  const int m = min(row, a.M - 1);  // rows past the last read the last
  f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int first = wv; first < KB; first += kMvAhead * kMvWaves) {
    if (first != wv) load(first);
#pragma unroll
    for (int i = 0; i < kMvAhead; ++i) {
      const int b = first + i * kMvWaves;
      if (b >= KB) break;
      i32x4 xr[2];
      float xsc;
      if constexpr (QUANT) {
        const uint8_t *from = room + m * stride + b * 128 + quarter * 16;
        const i32x4 *p = reinterpret_cast<const i32x4 *>(from);
        xr[0] = p[0];
        xr[1] = p[4];
        xsc = scales[m * KB + b];
      } else {
        const i32x4 *p = reinterpret_cast<const i32x4 *>(static_cast<const uint8_t *>(a.x) +
                                                         (size_t)m * K + b * 128 + quarter * 16);
        xr[0] = p[0];
        xr[1] = p[4];
        xsc = a.xs[(size_t)m * KB + b];
      }
      f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; c += 2)
          p = mfma_bf16(e4m3_bf16x8(wr[i][h][c], wr[i][h][c + 1]),
                        e4m3_bf16x8(xr[h][c], xr[h][c + 1]), p);
      const float sc = xsc * wsc[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(sc, p[e], acc[e]);
    }
  }

  // the waves' sums: [wave][row of x][weight row], a lane's four weight rows together
  if (QUANT) __syncthreads();  // the codes have been read
  float *const sums = reinterpret_cast<float *>(room);
  *reinterpret_cast<f32x4 *>(sums + (wv * 16 + row) * 16 + quarter * 4) = acc;
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * FEAT; i += kMvThreads) {
    const int f = i % FEAT, r = i / FEAT;
    if (r >= a.M || f >= a.N - n0) continue;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int v = 0; v < kMvWaves; ++v) {
      g += sums[v * 256 + r * 16 + f];
      if (GATEUP) u += sums[v * 256 + r * 16 + 8 + f];
    }
    const size_t o = (size_t)r * a.N + n0 + f;
    if (GATEUP)
      static_cast<float *>(a.y)[o] = swiglu(g, u);
    else if (a.f32)
      static_cast<float *>(a.y)[o] = g;
    else
      static_cast<uint16_t *>(a.y)[o] = f32_to_bf16_bits(g);
  }
}

template <int KIND, bool GATEUP>
static hipError_t mv_launch(const MatvecArgs &a, hipStream_t stream) {
  const dim3 grid(((unsigned)a.N + (GATEUP ? 7 : 15)) / (GATEUP ? 8 : 16)), block(kMvThreads);
  return launch(matvec_fp8_kernel<KIND, GATEUP>, grid, block, stream, a);
}

hipError_t launch_matvec_fp8(const MatvecArgs &a, hipStream_t stream) {
  if (a.w1) {
    if (a.xs) return mv_launch<kMvCodes, true>(a, stream);
    return mv_launch<kQbBf16, true>(a, stream);
  }
  if (a.xs) return mv_launch<kMvCodes, false>(a, stream);
  return a.x_f32 ? mv_launch<kQbF32, false>(a, stream) : mv_launch<kQbBf16, false>(a, stream);
}

}  // namespace moe

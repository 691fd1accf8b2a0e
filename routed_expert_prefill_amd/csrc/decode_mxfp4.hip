// Routed experts for single tokens: matrix-vector products with MXFP4
// weights (mx4.h), straight from the router's ids, in two launches and
// without route table, tile list or a combine of its own.
//
// At most 64 routes, so the whole routing fits one wave: lane r holds the
// expert of route r (or -1: masked, or an id outside [0, E)), and ballots
// find the routes that share an expert.  Each expert's weights are read once
// however many of its rows there are.
//
// Bound by that weight stream (a token of top-6 at d 4096, f 2048 reads
// 80 MB), so the kernels aim at bytes in flight: every wave issues all loads
// of up to eight steps of 128 columns (16 rows x 64 bytes per load, whole
// lines between two) into registers before it uses the first, and the
// activation rows go through LDS.  Products run on the 16x16x32 matrix
// instruction: its 16 columns hold the expert's rows (one, mostly); the
// matrix work is hidden behind the stream, and vector FMAs would leave less
// room for the decoding.  A lane's 16 bytes are 32 codes, one scale group;
// lane group c = l / 16 of a step holds group c, and MFMA j multiplies
// columns 8 j .. 8 j + 7 of all four groups.
#include "kernels.h"
#include "mx4.h"

namespace moe {

constexpr int kDecSteps = 8;   // steps of 128 columns whose loads a wave has in flight
constexpr int kDecRows = 4;    // activation rows a wave holds in LDS
constexpr int kDecCols = kDecSteps * 128;
constexpr int kDecRowBytes = kDecCols * 2 + 16;  // padded: rows start in different banks
constexpr int kDecGuWaves = 4;   // gate/up: the waves split the reduction
constexpr int kDecDnWaves = 16;  // down: the waves split experts and reduction

// The expert of route `lane`, or -1 if the route is not read.
__device__ __forceinline__ int dec_key(const DecodeArgs &a, int lane) {
  if (lane >= a.R) return -1;
  if (a.mask != nullptr && a.mask[lane] == 0) return -1;
  const int id = a.ids[lane];
  return id >= 0 && id < a.E ? id : -1;
}

__device__ __forceinline__ int dec_first(uint64_t set) { return __builtin_ctzll(set); }

__device__ __forceinline__ uint64_t dec_readlane64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

// One wave's products of TW weight tiles of 16 rows with up to kDecRows
// activation rows over steps [s0, s1): lane l holds weight row l % 16 of tile
// i at codes[i], scales[i] (row starts), activation row m starts at rows[m]
// for m < n.  acc[i] register r of lane l: weight row 4 (l / 16) + r,
// activation row l % 16 (repeated past n).
template <int TW>
__device__ __forceinline__ void dec_products(const uint8_t *const (&codes)[TW],
                                             const uint8_t *const (&scales)[TW],
                                             const uint16_t *const (&rows)[kDecRows], int n,
                                             int s0, int s1, uint8_t *lds, f32x4 (&acc)[TW]) {
  const int lane = lane_id();
  const int c = lane >> 4;
  const uint8_t *mine = lds + min(lane & 15, n - 1) * kDecRowBytes + c * 64;
  for (int s = s0; s < s1; s += kDecSteps) {
    const int steps = min(kDecSteps, s1 - s);
    // activation columns of these steps, 16 bytes per lane and load
    i32x4 xv[kDecRows][2];
#pragma unroll
    for (int m = 0; m < kDecRows; ++m) {
      if (m >= n) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int piece = lane + 64 * i;
        if (piece < steps * 16)
          xv[m][i] = *reinterpret_cast<const i32x4 *>(rows[m] + (size_t)s * 128 + piece * 8);
      }
    }
    // all weight loads; steps past the end load the last one again
    i32x4 raw[kDecSteps][TW];
    uint32_t sc[kDecSteps][TW];
#pragma unroll
    for (int i = 0; i < kDecSteps; ++i) {
      const size_t at = (size_t)min(s + i, s1 - 1);
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        raw[i][w] = *reinterpret_cast<const i32x4 *>(codes[w] + at * 64 + c * 16);
        sc[i][w] = *reinterpret_cast<const uint32_t *>(scales[w] + at * 4);
      }
    }
#pragma unroll
    for (int m = 0; m < kDecRows; ++m) {
      if (m >= n) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int piece = lane + 64 * i;
        if (piece < steps * 16)
          *reinterpret_cast<i32x4 *>(lds + m * kDecRowBytes + piece * 16) = xv[m][i];
      }
    }
#pragma unroll
    for (int i = 0; i < kDecSteps; ++i) {
      if (i >= steps) break;
      bf16x8 fx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        fx[j] = *reinterpret_cast<const bf16x8 *>(mine + i * 256 + j * 16);
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        const float scale = mx4_scale((sc[i][w] >> (8 * c)) & 0xffu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[w] = mfma_bf16(mx4_decode8((uint32_t)raw[i][w][j], scale), fx[j], acc[w]);
      }
    }
  }
}

// h[r, n0 .. n0 + 15] for every route r of one expert.  Workgroup (b, r): 16
// features of the expert of route r, if r is the first route with it.
__global__ __launch_bounds__(kDecGuWaves *kWave) void decode_gate_up_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t xs[kDecGuWaves][kDecRows * kDecRowBytes];
  __shared__ f32x4 part[kDecGuWaves][2][kWave];
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = blockIdx.x * 16, r0 = blockIdx.y;
  const int key = dec_key(a, lane);
  const int e = __builtin_amdgcn_readlane(key, r0);
  if (e < 0) return;
  uint64_t set = __ballot(key == e);
  if (dec_first(set) != r0) return;  // that route's workgroup has this one's rows
  const int steps = a.d / 128, per = (steps + kDecGuWaves - 1) / kDecGuWaves;
  const int s0 = min(wv * per, steps), s1 = min(s0 + per, steps);
  const size_t row = (size_t)e * a.f + n0 + (lane & 15);
  const uint8_t *codes[2] = {a.wg + row * (a.d / 2), a.wu + row * (a.d / 2)};
  const uint8_t *scales[2] = {a.sg + row * (a.d / 32), a.su + row * (a.d / 32)};
  while (set) {
    // the next rows of this expert
    const uint16_t *rows[kDecRows];
    int route[kDecRows], n = 0;
#pragma unroll
    for (int m = 0; m < kDecRows; ++m) {
      route[m] = 0;
      rows[m] = a.x;
      if (set) {
        route[m] = dec_first(set);
        rows[m] = a.x + (size_t)(route[m] / a.k) * a.d;
        set &= set - 1;
        ++n;
      }
    }
    f32x4 acc[2] = {};
    dec_products<2>(codes, scales, rows, n, s0, s1, xs[wv], acc);
    part[wv][0][lane] = acc[0];
    part[wv][1][lane] = acc[1];
    __syncthreads();
    // thread (wave g, lane l): the four features 4 (l / 16) .. + 3 of wave 0's
    // layout, feature g of them, row l % 16
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kDecGuWaves; ++w) {
      g += part[w][0][lane][wv];
      u += part[w][1][lane][wv];
    }
    const int m = lane & 15;
    if (m < n) {
      const int r = m == 0 ? route[0] : m == 1 ? route[1] : m == 2 ? route[2] : route[3];
      a.h[(size_t)r * a.f + n0 + 4 * (lane >> 4) + wv] = f32_to_bf16_bits(swiglu(g, u));
    }
    __syncthreads();  // part is written again
  }
}
static_assert(kDecGuWaves == 4 && kDecRows == 4, "the epilogue's mapping");

// out[t, n0 .. n0 + 15] for every token t.
__global__ __launch_bounds__(kDecDnWaves *kWave) void decode_down_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t hs[kDecDnWaves][kDecRows * kDecRowBytes];
  __shared__ f32x4 ys[2][kDecodeMaxRoutes][4];  // [half of the reduction][route][feature]
  __shared__ int read[kDecodeMaxRoutes];
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = blockIdx.x * 16;
  const int key = dec_key(a, lane);
  if (wv == 0) read[lane] = key >= 0;
  uint64_t same = 0;  // the routes with this lane's expert
  for (int r = 0; r < a.R; ++r) {
    const uint64_t b = __ballot(key == __builtin_amdgcn_readlane(key, r));
    if (lane == r) same = b;
  }
  uint64_t lead = __ballot(key >= 0 && dec_first(same) == lane);
  const int steps = a.f / 128, per = (steps + 1) / 2;
  int turn = 0;  // units (an expert, a half of the reduction) go round the waves
  while (lead) {
    const int r0 = dec_first(lead);
    lead &= lead - 1;
    const int e = __builtin_amdgcn_readlane(key, r0);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      if ((turn++ & (kDecDnWaves - 1)) != wv) continue;
      const int s0 = half ? per : 0, s1 = half ? steps : per;
      const size_t row = (size_t)e * a.d + n0 + (lane & 15);
      const uint8_t *codes[1] = {a.wd + row * (a.f / 2)};
      const uint8_t *scales[1] = {a.sd + row * (a.f / 32)};
      uint64_t set = dec_readlane64(same, r0);
      while (set) {
        const uint16_t *rows[kDecRows];
        int route[kDecRows], n = 0;
#pragma unroll
        for (int m = 0; m < kDecRows; ++m) {
          route[m] = 0;
          rows[m] = a.h;
          if (set) {
            route[m] = dec_first(set);
            rows[m] = a.h + (size_t)route[m] * a.f;
            set &= set - 1;
            ++n;
          }
        }
        f32x4 acc[1] = {};
        dec_products<1>(codes, scales, rows, n, s0, s1, hs[wv], acc);
        const int m = lane & 15;
        if (m < n) {
          const int r = m == 0 ? route[0] : m == 1 ? route[1] : m == 2 ? route[2] : route[3];
          ys[half][r][lane >> 4] = acc[0];
        }
      }
    }
  }
  __syncthreads();
  // the combine: routes of a token in ascending order from +0.0
  const int t = threadIdx.x >> 4, i = threadIdx.x & 15;
  if (t >= a.T) return;
  float sum = 0.0f;
  for (int j = 0; j < a.k; ++j) {
    const int r = t * a.k + j;
    if (read[r]) sum = __builtin_fmaf(a.w[r], ys[0][r][i >> 2][i & 3] + ys[1][r][i >> 2][i & 3], sum);
  }
  const size_t o = (size_t)t * a.d + n0 + i;
  if (a.shared) sum += a.shared[o];
  if (a.out) a.out[o] = sum;
  if (a.out_bf16) a.out_bf16[o] = f32_to_bf16_bits(sum);
}

hipError_t launch_decode_mx4(const DecodeArgs &a, hipStream_t stream) {
  hipLaunchKernelGGL(decode_gate_up_kernel, dim3(a.f / 16, a.R), dim3(kDecGuWaves * kWave), 0,
                     stream, a);
  hipLaunchKernelGGL(decode_down_kernel, dim3(a.d / 16), dim3(kDecDnWaves * kWave), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe

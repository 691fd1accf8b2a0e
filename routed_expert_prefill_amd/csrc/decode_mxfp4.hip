// Routed experts for single tokens: matrix-vector products with MXFP4
// weights (mx4.h), straight from the router's ids, in two launches and
// without route table, tile list or a combine of its own.
//
// At most 64 routes, so the whole routing fits one wave: lane r holds the
// expert of route r (or -1: masked, or an id outside [0, E)), and ballots
// find the routes that share an expert.  One pass over an expert's weights
// takes up to four of its routes in gate/up (kDecRows) and up to two in down,
// where a route has two rows; more routes take further passes, one after
// another, though the matrix instruction has 16 columns.
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
//
// MI355X, d 4096, f 2048, gate/up and down: one token of top-6 11.5 + 8.9 us
// (53.5 + 26.7 MB: 4.7 and 3.0 TB/s), four tokens, 21 experts, 40.5 + 22.6 us
// (4.6 and 4.1 TB/s).  At one token about 4 us of each launch are its start and
// the latency of its first loads.  Gate/up splits a reduction over four waves,
// which makes the workgroups of one token's six experts (768) fill the chip;
// down gives each wave whole experts, so that the routes' sums meet in LDS and
// no combine follows.
//
// h goes from one to the other as two bf16 numbers, the value rounded and what
// that took, rounded: 16 significant bits.  One rounding to bf16, as the grouped
// path has it, is as large as the output's own, and a token's few sums do not
// average it.  For experts of one or two routes the second part costs nothing
// (one token 20.4 -> 20.6 us, four tokens 63.9 -> 64.5); where more share an
// expert it halves the routes of a pass: 64 routes of one of 256 experts 150 us,
// 109 with h in one part.
#include "kernels.h"
#include "mx4.h"

namespace moe {

constexpr int kDecRows = 4;     // activation rows a wave holds in LDS
constexpr int kDecGuWaves = 4;  // gate/up: the waves split the reduction
constexpr int kDecDnWaves = 8;  // down: the waves split the experts
// steps of 128 columns whose loads a wave has in flight (with two weight
// tiles per step in gate/up, one in down)
constexpr int kDecGuSteps = 8;
constexpr int kDecDnSteps = 16;

// LDS of a wave for U steps and TW weight tiles: activation rows, then the
// weight rows' scales; both padded so that consecutive rows start in
// different banks.
template <int TW, int U>
struct DecLds {
  static constexpr int kRow = U * 256 + 16;
  static constexpr int kScales = U * 4 + 16;
  static constexpr int kBytes = kDecRows * kRow + TW * 16 * kScales;
};

// The expert of route `lane`, or -1 if the route is not read.
__device__ __forceinline__ int dec_key(const DecodeArgs &a, int lane) {
  const int r = min(lane, a.R - 1);
  const int id = a.ids[r];
  int on = 1;
  if (a.mask != nullptr) on = a.mask[r];
  return lane < a.R && on != 0 && id >= 0 && id < a.E ? id : -1;
}

__device__ __forceinline__ int dec_first(uint64_t set) { return __builtin_ctzll(set); }

__device__ __forceinline__ uint64_t dec_readlane64(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

// One wave's products of TW weight tiles of 16 rows with NR activation rows
// over U steps from step s: lane l holds weight row l % 16 of tile i at
// codes[i], scales[i] (row starts); activation row m starts at element
// rows[m] of x.  acc[i] register r of lane l: weight row 4 (l / 16) + r,
// activation row l % 16 (the last one again past NR).  lds: DecLds<TW, MU>
// of this wave, U <= MU.  Straight-line code, with every load issued ahead of the
// first wait: a branch between the steps lets the compiler sink each step's
// loads to it.
template <int TW, int MU, int NR, int U>
__device__ __forceinline__ void dec_steps(const uint8_t *const (&codes)[TW],
                                          const uint8_t *const (&scales)[TW], const uint16_t *x,
                                          const uint32_t (&rows)[kDecRows], int s, uint8_t *lds,
                                          f32x4 (&acc)[TW]) {
  using L = DecLds<TW, MU>;
  constexpr int XL = (U + 3) / 4;  // loads of 16 bytes per lane and activation row
  constexpr int SL = (U + 3) / 4;  // loads of scales: 4 bytes per step and weight row
  const int lane = lane_id();
  const int c = lane >> 4, row = lane & 15;
  i32x4 xv[NR][XL];
#pragma unroll
  for (int m = 0; m < NR; ++m)
#pragma unroll
    for (int i = 0; i < XL; ++i)
      xv[m][i] = *reinterpret_cast<const i32x4 *>(x + rows[m] + (size_t)s * 128 +
                                                  min(lane + 64 * i, U * 16 - 1) * 8);
  uint32_t sc[TW][SL];  // lane group c takes steps c, 4 + c, ..
#pragma unroll
  for (int w = 0; w < TW; ++w)
#pragma unroll
    for (int i = 0; i < SL; ++i)
      sc[w][i] = *reinterpret_cast<const uint32_t *>(scales[w] +
                                                     (size_t)(s + min(4 * i + c, U - 1)) * 4);
  i32x4 raw[U][TW];
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int w = 0; w < TW; ++w)
      raw[i][w] = *reinterpret_cast<const i32x4 *>(codes[w] + (size_t)(s + i) * 64 + c * 16);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int m = 0; m < NR; ++m)
#pragma unroll
    for (int i = 0; i < XL; ++i)
      *reinterpret_cast<i32x4 *>(lds + m * L::kRow + (lane + 64 * i) * 16) = xv[m][i];
  uint8_t *sc_lds = lds + kDecRows * L::kRow + row * L::kScales;
#pragma unroll
  for (int w = 0; w < TW; ++w)
#pragma unroll
    for (int i = 0; i < SL; ++i)
      *reinterpret_cast<uint32_t *>(sc_lds + w * 16 * L::kScales + (4 * i + c) * 4) = sc[w][i];
  i32x4 ss[TW][SL];
#pragma unroll
  for (int w = 0; w < TW; ++w)
#pragma unroll
    for (int i = 0; i < SL; ++i)
      ss[w][i] = *reinterpret_cast<const i32x4 *>(sc_lds + w * 16 * L::kScales + 16 * i);
  const uint8_t *mine = lds + min(row, NR - 1) * L::kRow + c * 64;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    bf16x8 fx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      fx[j] = *reinterpret_cast<const bf16x8 *>(mine + i * 256 + j * 16);
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      const float scale = mx4_scale(((uint32_t)ss[w][i >> 2][i & 3] >> (8 * c)) & 0xffu);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[w] = mfma_bf16(mx4_decode8((uint32_t)raw[i][w][j], scale), fx[j], acc[w]);
    }
  }
}

// The same over steps [s0, s1).
template <int TW, int MU, int NR>
__device__ __forceinline__ void dec_products_n(const uint8_t *const (&codes)[TW],
                                               const uint8_t *const (&scales)[TW],
                                               const uint16_t *x, const uint32_t (&rows)[kDecRows],
                                               int s0, int s1, uint8_t *lds, f32x4 (&acc)[TW]) {
  // many rows' activations take the registers of some of the steps
  constexpr int U = NR <= 2 ? MU : 4;
  int s = s0;
  for (; s + U <= s1; s += U) dec_steps<TW, MU, NR, U>(codes, scales, x, rows, s, lds, acc);
  if constexpr (U > 8) {
    if (s + 8 <= s1) {
      dec_steps<TW, MU, NR, 8>(codes, scales, x, rows, s, lds, acc);
      s += 8;
    }
  }
  if constexpr (U > 4) {
    if (s + 4 <= s1) {
      dec_steps<TW, MU, NR, 4>(codes, scales, x, rows, s, lds, acc);
      s += 4;
    }
  }
  if (s + 2 <= s1) {
    dec_steps<TW, MU, NR, 2>(codes, scales, x, rows, s, lds, acc);
    s += 2;
  }
  if (s < s1) dec_steps<TW, MU, NR, 1>(codes, scales, x, rows, s, lds, acc);
}

// The same for n = 1 .. kDecRows activation rows; rows past n repeat one.  ONE
// is the n that single rows of an expert come with (gate/up: 1, down: 2).
// A row's sums do not depend on n: the steps are taken in one order.
template <int TW, int MU, int ONE>
__device__ __forceinline__ void dec_products(const uint8_t *const (&codes)[TW],
                                             const uint8_t *const (&scales)[TW], const uint16_t *x,
                                             const uint32_t (&rows)[kDecRows], int n, int s0,
                                             int s1, uint8_t *lds, f32x4 (&acc)[TW]) {
  if (n == ONE)
    dec_products_n<TW, MU, ONE>(codes, scales, x, rows, s0, s1, lds, acc);
  else
    dec_products_n<TW, MU, kDecRows>(codes, scales, x, rows, s0, s1, lds, acc);
}

// The next N of an expert's routes `set`, which loses them; past the result's
// count they repeat the first.
template <int N>
__device__ __forceinline__ int dec_next_routes(uint64_t &set, int (&route)[N]) {
  int n = 0;
#pragma unroll
  for (int m = 0; m < N; ++m) {
    route[m] = route[0];
    if (m == 0 || set) {
      route[m] = dec_first(set);
      set &= set - 1;
      ++n;
    }
  }
  return n;
}

// h[r, n0 .. n0 + 15] for every route r of one expert.  Workgroup (b, r): 16
// features of the expert of route r, if r is the first route with it.
__global__ __launch_bounds__(kDecGuWaves *kWave) void decode_gate_up_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kDecGuWaves][DecLds<2, kDecGuSteps>::kBytes];
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
    int route[kDecRows];
    const int n = dec_next_routes(set, route);
    uint32_t rows[kDecRows];
#pragma unroll
    for (int m = 0; m < kDecRows; ++m) rows[m] = (uint32_t)(route[m] / a.k) * (uint32_t)a.d;
    f32x4 acc[2] = {};
    dec_products<2, kDecGuSteps, 1>(codes, scales, a.x, rows, n, s0, s1, lds[wv], acc);
    // the waves' parts of the sums, where their activation rows were
    f32x4 *part = reinterpret_cast<f32x4 *>(lds[wv]);
    part[lane] = acc[0];
    part[kWave + lane] = acc[1];
    __syncthreads();
    // wave g, lane l: feature 4 (l / 16) + g of activation row l % 16
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kDecGuWaves; ++w) {
      const float *p = reinterpret_cast<const float *>(lds[w]) + lane * 4 + wv;
      g += p[0];
      u += p[kWave * 4];
    }
    const int m = lane & 15;
    if (m < n) {
      const int r = m == 0 ? route[0] : m == 1 ? route[1] : m == 2 ? route[2] : route[3];
      const size_t at = (size_t)r * a.f + n0 + 4 * (lane >> 4) + wv;
      const float v = swiglu(g, u);
      const uint16_t top = f32_to_bf16_bits(v);
      a.h[at] = top;
      // what rounding took, rounded; nothing beside an infinity or a NaN
      const bool finite = (top & 0x7f80u) != 0x7f80u;
      a.h[(size_t)a.R * a.f + at] =
          finite ? f32_to_bf16_bits(v - bf16_bits_to_f32(top)) : (uint16_t)0;
    }
    __syncthreads();  // the parts make room for the next rows
  }
}
static_assert(kDecGuWaves == 4 && kDecRows == 4, "the epilogues' mapping");

// out[t, n0 .. n0 + 15] for every token t: the experts go round the waves,
// and the routes' sums meet in LDS.
__global__ __launch_bounds__(kDecDnWaves *kWave) void decode_down_kernel(DecodeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t
      lds[kDecDnWaves][DecLds<1, kDecDnSteps>::kBytes];
  __shared__ f32x4 ys[kDecodeMaxRoutes][4];  // [route][feature]
  __shared__ int read[kDecodeMaxRoutes];
  __shared__ float gate[kDecodeMaxRoutes];
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n0 = blockIdx.x * 16;
  const int key = dec_key(a, lane);
  if (wv == 0) {  // for the combine, whose loads would otherwise wait in a row
    read[lane] = key >= 0;
    gate[lane] = a.w[min(lane, a.R - 1)];
  }
  uint64_t same = 0;  // the routes with this lane's expert
  for (int r = 0; r < a.R; ++r) {
    const uint64_t b = __ballot(key == __builtin_amdgcn_readlane(key, r));
    if (lane == r) same = b;
  }
  uint64_t lead = __ballot(key >= 0 && dec_first(same) == lane);
  const int steps = a.f / 128;
  for (int turn = 0; lead; ++turn) {
    const int r0 = dec_first(lead);
    lead &= lead - 1;
    if ((turn & (kDecDnWaves - 1)) != wv) continue;
    const size_t row = (size_t)__builtin_amdgcn_readlane(key, r0) * a.d + n0 + (lane & 15);
    const uint8_t *codes[1] = {a.wd + row * (a.f / 2)};
    const uint8_t *scales[1] = {a.sd + row * (a.f / 32)};
    uint64_t set = dec_readlane64(same, r0);
    while (set) {
      // rows 2 m and 2 m + 1: the two parts of h of route m
      int route[kDecRows / 2];
      const int n = dec_next_routes(set, route);
      uint32_t rows[kDecRows];
#pragma unroll
      for (int m = 0; m < kDecRows; ++m)
        rows[m] = (uint32_t)(route[m / 2] + (m % 2) * a.R) * (uint32_t)a.f;
      f32x4 acc[1] = {};
      dec_products<1, kDecDnSteps, 2>(codes, scales, a.h, rows, 2 * n, 0, steps, lds[wv], acc);
      f32x4 y;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float rest = __shfl_xor(acc[0][i], 1);
        y[i] = acc[0][i];
        // an infinite weight has made the first part's sum what it is, and times
        // the second part (zero, or of the other sign) it would make it NaN
        if (fabsf(y[i]) < __builtin_inff()) y[i] += rest;
      }
      const int m = lane & 15;
      if (m % 2 == 0 && m / 2 < n) ys[m == 0 ? route[0] : route[1]][lane >> 4] = y;
    }
  }
  __syncthreads();
  // the combine: routes of a token in ascending order from +0.0
  for (int o = threadIdx.x; o < a.T * 16; o += kDecDnWaves * kWave) {
    const int t = o >> 4, i = o & 15;
    const size_t at = (size_t)t * a.d + n0 + i;
    float sum = 0.0f, sh = 0.0f;
    if (a.shared) sh = a.shared[at];
    for (int r = t * a.k; r < (t + 1) * a.k; ++r)
      if (read[r]) sum = __builtin_fmaf(gate[r], ys[r][i >> 2][i & 3], sum);
    if (a.shared) sum += sh;
    if (a.out) a.out[at] = sum;
    if (a.out_bf16) a.out_bf16[at] = f32_to_bf16_bits(sum);
  }
}

hipError_t launch_decode_mx4(const DecodeArgs &a, hipStream_t stream) {
  const hipError_t err =
      launch(decode_gate_up_kernel, dim3(a.f / 16, a.R), dim3(kDecGuWaves * kWave), stream, a);
  if (err != hipSuccess) return err;
  return launch(decode_down_kernel, dim3(a.d / 16), dim3(kDecDnWaves * kWave), stream, a);
}

}  // namespace moe

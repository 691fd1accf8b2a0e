// Residual addition and root-mean-square norm of the rows ahead of a layer,
// with the normalised rows in bf16 and / or quantised to E4M3 with one scale
// per row:
//
//   v = residual + x,  r = 1 / sqrt(mean(v^2) + eps),  n = (v * weight) * r
//   residual_out = v,  y = bf16(n),  s = max|n| / 448,  q = e4m3(n / s)
//
// A row is read once and stays in registers as fp32; each output is rounded
// once from it (n is not rounded to bf16 ahead of the quantisation, and the
// norm takes v as it is before residual_out is rounded).  The squares are
// summed in fp64: rows whose squares overflow fp32 keep their norm, and the
// fp64 work (one conversion and one FMA per element) hides behind the memory
// traffic.  max|n| needs no second pass: rounding is monotone, so
// max|n| = fl(max|v * weight| * r), and both reductions share one exchange.
//
// Bound by memory traffic (9 bytes per element with bf16 rows, a bf16
// residual and both outputs) from a few hundred rows on, by the latency of one row's load,
// reduction and store below that.
#include "e4m3.h"
#include "kernels.h"

namespace moe {

constexpr int kNmThreads = 256;
constexpr int kNmWaves = kNmThreads / kWave;
constexpr int kNmMaxChunks = 8;  // 8-element chunks per thread
constexpr int kNmMaxCols = kNmThreads * 8 * kNmMaxChunks;  // 16384

// Eight consecutive elements as loaded: bf16 in one register quad, fp32 in two.
template <bool F32>
struct NmRaw {
  i32x4 a[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void *base, size_t i) {
    if constexpr (F32) {
      const i32x4 *p = reinterpret_cast<const i32x4 *>(static_cast<const float *>(base) + i);
      a[0] = p[0];
      a[1] = p[1];
    } else {
      a[0] = *reinterpret_cast<const i32x4 *>(static_cast<const uint16_t *>(base) + i);
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (F32) {
      return __int_as_float(a[e >> 2][e & 3]);
    } else {
      const uint32_t two = (uint32_t)a[0][e >> 1];
      return __uint_as_float((e & 1) ? two & 0xffff0000u : two << 16);
    }
  }
};

__device__ __forceinline__ void nm_store8(void *base, size_t i, bool f32, const float (&v)[8]) {
  if (f32) {
    f32x4 *p = reinterpret_cast<f32x4 *>(static_cast<float *>(base) + i);
    p[0] = f32x4{v[0], v[1], v[2], v[3]};
    p[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    i32x4 o;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      o[w] = (int)((uint32_t)f32_to_bf16_bits(v[2 * w]) |
                   ((uint32_t)f32_to_bf16_bits(v[2 * w + 1]) << 16));
    *reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(base) + i) = o;
  }
}

__device__ __forceinline__ double nm_wave_sum(double v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ float nm_wave_max(float v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}

// 1 / sqrt(m): in fp32 where m is well inside its range, in fp64 elsewhere.
__device__ __forceinline__ float nm_rsqrt(double m) {
  if (m > 1e-30 && m < 1e38) return 1.0f / sqrtf((float)m);
  return (float)(1.0 / sqrt(m));
}

// NC 8-element chunks per thread.  WIDE: the whole workgroup takes one row;
// otherwise each of its waves takes a row of its own.
// XF: x is fp32 (else bf16).  RES: 0 no residual, 1 bf16, 2 fp32.
template <int NC, bool WIDE, bool XF, int RES>
__global__ __launch_bounds__(kNmThreads) void add_rmsnorm_kernel(NormArgs a) {
  constexpr int TPR = WIDE ? kNmThreads : kWave;  // threads per row
  __shared__ double part_sum[kNmWaves];
  __shared__ float part_max[kNmWaves];
  const int wave = threadIdx.x / kWave;
  const int tid = WIDE ? (int)threadIdx.x : lane_id();
  const int row = WIDE ? (int)blockIdx.x : (int)blockIdx.x * kNmWaves + wave;
  if (!WIDE && row >= a.rows) return;  // no barrier below without WIDE
  const size_t base = (size_t)row * a.d;

  NmRaw<XF> xr[NC];
  NmRaw<RES == 2> rr[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = (c * TPR + tid) * 8;
    if (i < a.d) {
      xr[c].load(a.x, base + i);
      if (RES) rr[c].load(a.residual, base + i);
    }
  }
  float v[NC][8], n[NC][8];
  double sum = 0.0;
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = (c * TPR + tid) * 8;
    if (i >= a.d) continue;
    float w[8];
    if (a.w_f32) {
      NmRaw<true> wr;
      wr.load(a.weight, i);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = wr.at(e);
    } else {
      NmRaw<false> wr;
      wr.load(a.weight, i);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = wr.at(e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[c][e] = xr[c].at(e);
      if (RES) v[c][e] += rr[c].at(e);
      const double t = (double)v[c][e];
      sum = __builtin_fma(t, t, sum);
      n[c][e] = v[c][e] * w[e];
      top = fmaxf(top, fabsf(n[c][e]));
    }
    if (a.residual_out) nm_store8(a.residual_out, base + i, RES == 2 || (RES == 0 && XF), v[c]);
  }
  sum = nm_wave_sum(sum);
  top = nm_wave_max(top);
  if (WIDE) {
    if (lane_id() == 0) {
      part_sum[wave] = sum;
      part_max[wave] = top;
    }
    __syncthreads();
    sum = part_sum[0];
    top = part_max[0];
#pragma unroll
    for (int w = 1; w < kNmWaves; ++w) {
      sum += part_sum[w];
      top = fmaxf(top, part_max[w]);
    }
  }
  const float r = nm_rsqrt(sum / a.d + (double)a.eps);
  top *= r;
  const bool zero = top == 0.0f;
  const float sc = q_scale(top);
  bool exact;
  const float rcp = quant_rcp(sc, &exact);
  if (a.s && tid == 0) a.s[row] = sc;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = (c * TPR + tid) * 8;
    if (i >= a.d) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) n[c][e] *= r;
    if (a.y) nm_store8(a.y, base + i, false, n[c]);
    if (a.q) {
      const float lo[4] = {n[c][0], n[c][1], n[c][2], n[c][3]};
      const float hi[4] = {n[c][4], n[c][5], n[c][6], n[c][7]};
      uint2 o;
      o.x = quant_e4m3_x4(lo, sc, rcp, exact, zero);
      o.y = quant_e4m3_x4(hi, sc, rcp, exact, zero);
      *reinterpret_cast<uint2 *>(a.q + base + i) = o;
    }
  }
}

int norm_max_cols() { return kNmMaxCols; }

template <int NC, bool WIDE>
static void nm_launch(const NormArgs &a, hipStream_t stream) {
  const dim3 grid(WIDE ? a.rows : (a.rows + kNmWaves - 1) / kNmWaves), block(kNmThreads);
#define MOE_NORM_CASE(XF, RES)                                                          \
  if (a.x_f32 == XF && a.res_kind == RES) {                                             \
    hipLaunchKernelGGL((add_rmsnorm_kernel<NC, WIDE, XF, RES>), grid, block, 0, stream, a); \
    return;                                                                             \
  }
  MOE_NORM_CASE(false, 0) MOE_NORM_CASE(false, 1) MOE_NORM_CASE(false, 2)
  MOE_NORM_CASE(true, 0) MOE_NORM_CASE(true, 1) MOE_NORM_CASE(true, 2)
#undef MOE_NORM_CASE
}

hipError_t launch_add_rmsnorm(const NormArgs &a, hipStream_t stream) {
  const int per = kNmThreads * 8;  // elements of one chunk of every thread of a workgroup
  if (a.d <= kWave * 8)
    nm_launch<1, false>(a, stream);
  else if (a.d <= per)
    nm_launch<1, true>(a, stream);
  else if (a.d <= 2 * per)
    nm_launch<2, true>(a, stream);
  else if (a.d <= 4 * per)
    nm_launch<4, true>(a, stream);
  else
    nm_launch<8, true>(a, stream);
  return hipGetLastError();
}

}  // namespace moe

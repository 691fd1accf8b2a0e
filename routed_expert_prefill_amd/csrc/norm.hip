// Residual addition and root-mean-square norm of the rows ahead of a layer,
// with the normalised rows in bf16 and / or quantised to E4M3 with one scale
// per row:
//
//   v = residual + x,  r = 1 / sqrt(mean(v^2) + eps),  n = (v * weight) * r
//   residual_out = v,  y = bf16(n),  s = max|n| / 448,  q = e4m3(n / s)
//
// A row is read once and stays in registers; each output is rounded once (n
// is not rounded to bf16 ahead of the quantisation, and the norm takes v as it
// is before residual_out is rounded).  The squares are summed in fp64: rows
// whose squares overflow fp32 keep their norm.
//
// Codes.  n / s = v weight 448 / max|v weight|: the root cancels, and the
// codes are those of that quotient in fp64.  Nearly every element takes its
// code from fp32: y = n (1 / s) lies within 8 x 2^-24 of the quotient (v, two
// products, s with its product and division, its reciprocal, and the product
// with it: one rounding each), so where no midpoint between two codes is near,
// the code is the same; the few others are formed again from the inputs in
// fp64.  Codes taken from fp32 alone were off by one step in about one element
// of a million.
//
// A wave whose products v weight leave fp32, or whose root is far from 1, forms
// n in fp64, and a row's scale with it.  That it has to costs a maximum for
// each element that keeps NaN (which the row's own maximum drops), 0.1 to 0.4 us
// a call: 401 rows of 4096 8.0 -> 8.2, 8192 rows 49.4 -> 50.4.
//
// Bound by memory traffic (9 bytes per element with bf16 rows, a bf16
// residual and both outputs) from a few thousand rows on: 8192 rows of 4096 take
// 58.5 us on MI355X, 5.2 TB/s, where a large copy reaches 4.8.  Below that by
// the latency of one row's loads, reduction and stores: one row of 4096 4 us, 401
// rows 8 to 9 us against 3 us of traffic.  Rows of several chunks a thread wait
// for a store of their own in between: the weight of the next chunk is loaded
// behind residual_out's store, and stores count among the loads that the wait
// for it covers.  A workgroup to a row keeps the latency short; rows of up to
// 512 columns would leave three of its waves idle, so a wave takes one there.
#include "e4m3.h"
#include "kernels.h"

namespace moe {

constexpr int kNmThreads = 256;
constexpr int kNmWaves = kNmThreads / kWave;
// Workgroups in x: a grid takes fewer than 2^32 threads in each dimension.
constexpr unsigned kNmLine = 1u << 22;
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

// Stores past the caches (nontemporal): nothing here reads a line again, and
// dirty lines left in L2 are what the kernel's end waits for (8192 rows of
// 4096: 67 -> 59.5 us, 1999 rows of 1416: 12 -> 10.4).  Loads gained nothing.
__device__ __forceinline__ void nm_store8(void *base, size_t i, bool f32, const float (&v)[8]) {
  if (f32) {
    f32x4 *p = reinterpret_cast<f32x4 *>(static_cast<float *>(base) + i);
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
  } else {
    i32x4 o;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      o[w] = (int)((uint32_t)f32_to_bf16_bits(v[2 * w]) |
                   ((uint32_t)f32_to_bf16_bits(v[2 * w + 1]) << 16));
    __builtin_nontemporal_store(o, reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(base) + i));
  }
}

__device__ __forceinline__ double nm_wave_sum(double v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// The largest of the lanes' magnitudes, NaN if a lane has `none` (fmax drops it).
__device__ __forceinline__ double nm_wave_max(double v, bool none) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v = fmax(v, __shfl_xor(v, m));
  return __any(none) ? __builtin_nan("") : v;
}

// The same of two.
__device__ __forceinline__ double nm_max(double a, double b) { return b > a || b != b ? b : a; }

// Whether a value within 8 x 2^-24 of y may have another code than y: it is
// near a midpoint between codes, which are the patterns with low bits 0x80000
// in the normal range and odd multiples of 2^-10 below it, or no number.
__device__ __forceinline__ bool nm_near_midpoint(float y) {
  const uint32_t a = __float_as_uint(y) & 0x7fffffffu;
  const float t = __uint_as_float(a) * 512.0f;
  return a >= 0x3c800000u ? a > 0x7f800000u || ((a & 0xfffffu) - 0x7fff0u) < 32u
                          : fabsf(t - floorf(t) - 0.5f) < 1e-5f;
}

// E4M3 code of a fp64 value, rounded once: fp32 rounded to odd on the way.
__device__ __forceinline__ uint32_t nm_code(double t) {
  uint32_t b = __float_as_uint((float)t);
  const double f = fabs((double)__uint_as_float(b));
  if (f > fabs(t)) --b;
  if (f != fabs(t)) b |= 1u;
  return f32_to_e4m3(__uint_as_float(b));
}

// NC 8-element chunks per thread.  WIDE: the whole workgroup takes one row;
// otherwise each of its waves takes a row of its own.
// XF: x is fp32 (else bf16).  RES: 0 no residual, 1 bf16, 2 fp32.
template <int NC, bool WIDE, bool XF, int RES>
__global__ __launch_bounds__(kNmThreads) void add_rmsnorm_kernel(NormArgs a) {
  constexpr int TPR = WIDE ? kNmThreads : kWave;  // threads per row
  __shared__ double part_sum[kNmWaves];
  __shared__ double part_max[kNmWaves];
  const int wave = threadIdx.x / kWave;
  const int tid = WIDE ? (int)threadIdx.x : lane_id();
  // the last line of workgroups may end past the rows
  const unsigned block = blockIdx.y * kNmLine + blockIdx.x;
  if (WIDE && block >= (unsigned)a.rows) return;
  const int row = WIDE ? (int)block : (int)(block * kNmWaves) + wave;
  if (!WIDE && (row < 0 || row >= a.rows)) return;  // no barrier below without WIDE
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
  // element e of chunk c of x + residual, unrounded
  const auto sum_of = [&](int c, int e) {
    return RES ? (double)xr[c].at(e) + (double)rr[c].at(e) : (double)xr[c].at(e);
  };
  const auto weight_at = [&](int i) {
    return a.w_f32 ? static_cast<const float *>(a.weight)[i]
                   : bf16_bits_to_f32(static_cast<const uint16_t *>(a.weight)[i]);
  };
  float n[NC][8];
  double sum = 0.0, top = 0.0;
  float ptop = 0.0f;  // largest |v weight| of this thread in fp32, NaN if one is
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
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = xr[c].at(e);
      if (RES) v[e] += rr[c].at(e);
      const double t = (double)v[e];
      sum = __builtin_fma(t, t, sum);
      n[c][e] = v[e] * w[e];
      if (a.q) top = fmax(top, fabs(sum_of(c, e) * (double)w[e]));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ptop = __builtin_elementwise_maximum(ptop, fabsf(n[c][e]));
    if (a.residual_out) nm_store8(a.residual_out, base + i, RES == 2 || (RES == 0 && XF), v);
  }
  sum = nm_wave_sum(sum);
  top = nm_wave_max(top, ptop != ptop);
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
      top = nm_max(top, part_max[w]);
    }
  }
  const double m = sum / a.d + (double)a.eps;
  float amax, sc, rcp = 0.0f;
  bool exact;
  // Where fp32 may not do.  For n = (v weight) r: with a product of this wave
  // beyond the largest number (or none), or a root far from 1.  (A subnormal product is off
  // by at most 2^-150 r in n: with r below 2^12 an eighth of half a step of the
  // smallest normal bf16.)  For the scale: with largest products near an end too.
  const bool ends = __any(!(ptop <= 3.40282347e38f) || !(m > 6e-8 && m < 1e38));
  if (ends || __any(a.q && !(top >= 1e-28 && top <= 1e38))) {
    const double rd = 1.0 / sqrt(m);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = (c * TPR + tid) * 8;
      if (i >= a.d) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = xr[c].at(e);
        if (RES) v += rr[c].at(e);
        n[c][e] = ends ? (float)((double)v * (double)weight_at(i + e) * rd)
                       : n[c][e] * (1.0f / sqrtf((float)m));
      }
    }
    // a v beyond fp32 is an infinity there, and its n then NaN, whatever top is
    const double t = sum < __builtin_inf() ? top * rd : __builtin_nan("");
    amax = (float)t;
    sc = amax == 0.0f ? 1.0f : (float)(t * (1.0 / 448.0));
    exact = true;
  } else {
    const float r = 1.0f / sqrtf((float)m);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) n[c][e] *= r;
    amax = (float)top * r;
    sc = q_scale(amax);
    rcp = quant_rcp(sc, &exact);
  }
  if (a.s && tid == 0) a.s[row] = sc;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int i = (c * TPR + tid) * 8;
    if (i >= a.d) continue;
    if (a.y) nm_store8(a.y, base + i, false, n[c]);
    if (!a.q) continue;
    uint2 o = {};
    if (amax != 0.0f) {
      bool any = exact;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[c][e] *= rcp;
        any = any || nm_near_midpoint(n[c][e]);
      }
      o.x = cvt_e4m3_x2<true>(n[c][2], n[c][3], cvt_e4m3_x2<false>(n[c][0], n[c][1], 0u));
      o.y = cvt_e4m3_x2<true>(n[c][6], n[c][7], cvt_e4m3_x2<false>(n[c][4], n[c][5], 0u));
      if (any) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (!exact && !nm_near_midpoint(n[c][e])) continue;
          const double t = sum_of(c, e) * (double)weight_at(i + e) * 448.0 / top;
          const uint32_t code = nm_code(sc == sc ? t : (double)sc);
          uint32_t &part = e < 4 ? o.x : o.y;
          part = (part & ~(0xffu << (8 * (e & 3)))) | (code << (8 * (e & 3)));
        }
      }
    }
    __builtin_nontemporal_store((uint64_t)o.x | (uint64_t)o.y << 32, reinterpret_cast<uint64_t *>(a.q + base + i));
  }
}

int norm_max_cols() { return kNmMaxCols; }

template <int NC, bool WIDE>
static hipError_t nm_launch(const NormArgs &a, hipStream_t stream) {
  const unsigned blocks = WIDE ? (unsigned)a.rows : ((unsigned)a.rows + kNmWaves - 1) / kNmWaves;
  const dim3 grid(blocks < kNmLine ? blocks : kNmLine, (blocks + kNmLine - 1) / kNmLine),
      block(kNmThreads);
#define MOE_NORM_CASE(XF, RES)             \
  if (a.x_f32 == XF && a.res_kind == RES) \
    return launch(add_rmsnorm_kernel<NC, WIDE, XF, RES>, grid, block, stream, a);
  MOE_NORM_CASE(false, 0) MOE_NORM_CASE(false, 1) MOE_NORM_CASE(false, 2)
  MOE_NORM_CASE(true, 0) MOE_NORM_CASE(true, 1) MOE_NORM_CASE(true, 2)
#undef MOE_NORM_CASE
  return hipErrorInvalidValue;  // the C ABI passes the kinds above only
}

hipError_t launch_add_rmsnorm(const NormArgs &a, hipStream_t stream) {
  const int per = kNmThreads * 8;  // elements of one chunk of every thread of a workgroup
  if (a.d <= kWave * 8) return nm_launch<1, false>(a, stream);
  if (a.d <= per) return nm_launch<1, true>(a, stream);
  if (a.d <= 2 * per) return nm_launch<2, true>(a, stream);
  if (a.d <= 4 * per) return nm_launch<4, true>(a, stream);
  return nm_launch<8, true>(a, stream);
}

}  // namespace moe

// Product of E4M3 rows with E4M3 weights, a scale for each block of 128:
//
//   y[m, n] = sum over blocks b of 128 columns of
//             (xs[m, b] * ws[n / 128, b]) * sum over c in b of x[m, c] * w[n, c]
//
// A block's sum is a chain of matrix instructions from zero, folded into the fp32
// accumulator once with the product of the two scales in fp32.
//
// fp32 results: codes are turned into bf16, which holds every one of them, and go
// through the 32x32x16 bf16 instruction.  The 8-bit instructions (both the 32x32x64
// and the 32x32x16 one) align the products of eight neighbouring columns to the
// largest of the eight and drop what lies more than 13 bits below it, seen on
// MI355X with single products beside a large one: over random codes their sums
// are 1.5e-5 of the result's norm off, where fp32's are 1e-7 to 1e-6.  bf16
// results, whose own rounding is 1.7e-3, take the 8-bit 32x32x64 one, twice as fast.
//
// A workgroup computes BM rows by BN weight rows.  A stage of its LDS ring
// (ring.h) is one block of 128 columns: a 128-byte line of each row, and the
// rows' scales for that block.
#include "kernels.h"
#include "ring.h"

namespace moe {

constexpr int kMmThreads = 512;
constexpr int kMmWaves = kMmThreads / kWave;
constexpr int kMmLds = 160 * 1024;
// Workgroups in x: a grid takes fewer than 2^32 threads in each dimension.
constexpr unsigned kMmLine = 1u << 22;

__device__ __forceinline__ f32x16 mm_mfma(const i32x8 &a, const i32x8 &b, const f32x16 &c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
}

// Eight E4M3 codes as bf16, which holds each of them.
__device__ __forceinline__ bf16x8 mm_bf16(int lo, int hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ i32x8 mm_lds(const uint8_t *p0, const uint8_t *p1) {
  const i32x4 lo = *reinterpret_cast<const i32x4 *>(p0);
  const i32x4 hi = *reinterpret_cast<const i32x4 *>(p1);
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// 16 (4) bytes per lane from base + off into LDS at lds_byte_addr + 16 (4) * lane;
// inline for the reason that dma16 is.
__device__ __forceinline__ void mm_dma16(uint32_t off, const void *base, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_byte_addr)
               : "memory");
}
__device__ __forceinline__ void mm_dma4(uint32_t off, const void *base, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_byte_addr)
               : "memory");
}

// WM x WN waves, each TT x TW tiles of 32 x 32.
template <int BM, int BN, int WM>
struct MmTile {
  static constexpr int kWN = kMmWaves / WM;
  static constexpr int kTT = BM / 32 / WM, kTW = BN / 32 / kWN;
  static_assert(kTT * WM * 32 == BM && kTW * kWN * 32 == BN, "whole tiles to every wave");
  static constexpr int kRowLoads = (BM + BN) / 8;       // of 8 rows
  static constexpr int kScaleLoads = (BM + 63) / 64;    // of 64 rows
  static constexpr int kLoads = kRowLoads + kScaleLoads;
  static constexpr int kSlot = kRowLoads * 1024 + kScaleLoads * 256;
  static constexpr int kDepth = kMmLds / kSlot < 6 ? kMmLds / kSlot : 6;
  static_assert(kDepth >= 2, "one stage loads while one is read");
};

template <int BM, int BN, int WM, bool F32>
__global__ __launch_bounds__(kMmThreads, 1) void matmul_fp8_kernel(MatmulArgs a) {
  using L = MmTile<BM, BN, WM>;
  constexpr int TT = L::kTT, TW = L::kTW, NS = L::kDepth, SLOT = L::kSlot;
  constexpr int MAXJ = (L::kLoads + kMmWaves - 1) / kMmWaves;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NS * SLOT];
  const uint32_t ring_lds = lds_addr(ring);
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int tiles_n = (a.N + BN - 1) / BN;
  const unsigned tile = blockIdx.y * kMmLine + blockIdx.x;
  const int tm = (int)(tile / (unsigned)tiles_n), tn = (int)(tile % (unsigned)tiles_n);
  if ((long long)tm * BM >= a.M) return;  // the last line of workgroups may end past the tiles
  const int m0 = tm * BM, n0 = tn * BN;
  const int K = a.K, nst = K / 128;

  // load i fills stage rows 8 i .. 8 i + 7 (rows past the last read the last);
  // the loads behind them fill the rows' scales
  const int lr = lane >> 3;
  const uint8_t *xb = a.x + (size_t)m0 * K, *wb = a.w + (size_t)n0 * K;
  const float *sb = a.xs + (size_t)m0 * nst;
  uint32_t off[MAXJ];
#pragma unroll
  for (int j = 0; j < MAXJ; ++j) {
    const int i = wv + kMmWaves * j;
    const int chunk = ring_slot(i * 8 + lr, lane & 7) * 16;
    off[j] = 0;
    if (i < BM / 8)
      off[j] = (uint32_t)min(i * 8 + lr, a.M - 1 - m0) * (uint32_t)K + chunk;
    else if (i < L::kRowLoads)
      off[j] = (uint32_t)min((i - BM / 8) * 8 + lr, a.N - 1 - n0) * (uint32_t)K + chunk;
    else if (i < L::kLoads)
      off[j] = (uint32_t)min((i - L::kRowLoads) * 64 + lane, a.M - 1 - m0) * (uint32_t)nst * 4u;
  }
  const int cnt = (L::kLoads - wv + kMmWaves - 1) / kMmWaves;  // loads of this wave in a stage
  auto issue = [&](int s, int slot) {
    const uint32_t base = ring_lds + (uint32_t)(slot * SLOT);
#pragma unroll
    for (int j = 0; j < MAXJ; ++j) {
      const int i = wv + kMmWaves * j;
      if (i < BM / 8)
        mm_dma16(off[j], xb + (size_t)s * 128, base + (uint32_t)i * 1024u);
      else if (i < L::kRowLoads)
        mm_dma16(off[j], wb + (size_t)s * 128, base + (uint32_t)i * 1024u);
      else if (i < L::kLoads)
        mm_dma4(off[j], sb + s,
                base + (uint32_t)(L::kRowLoads * 1024 + (i - L::kRowLoads) * 256));
    }
  };

  // this wave's tiles, and the scales of its weight rows' blocks: those of 64
  // stages are held by the lanes.  (Loaded stage by stage they would have the
  // compiler wait for every load in flight, the ring's included.)
  const int at0 = wv / L::kWN * TT, wt0 = wv % L::kWN * TW;
  float held[TW];
  auto hold = [&](int s) {
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
      held[tw] = a.ws[(size_t)(min(n0 + (wt0 + tw) * 32, a.N - 1) / 128) * nst +
                      min(s + lane, nst - 1)];
  };
  hold(0);

  // reader: row (lane & 31) of a 32-row tile; 64-element step ks takes the
  // chunks 4 ks + 2 (lane >> 5) and the next
  const int rr = lane & 31, rh = lane >> 5;
  int off0[2], off1[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    off0[ks] = rr * 128 + ring_slot(rr, 4 * ks + 2 * rh) * 16;
    off1[ks] = rr * 128 + ring_slot(rr, 4 * ks + 2 * rh + 1) * 16;
  }
  f32x16 acc[TT][TW];
#pragma unroll
  for (int tt = 0; tt < TT; ++tt)
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[tt][tw][j] = 0.f;

#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nst) issue(s, s);
  int slot = 0;
  for (int s = 0; s < nst; ++s) {
    if (s != 0 && s % kWave == 0) hold(s);
    wait_vm(cnt * min(NS - 2, nst - 1 - s));
    ring_barrier();  // stage s is in LDS for everyone; stage s - 1 is consumed
    const int ahead = s + NS - 1;
    if (ahead < nst) issue(ahead, slot == 0 ? NS - 1 : slot - 1);
    const uint8_t *buf = ring + slot * SLOT;
    const float *xsc = reinterpret_cast<const float *>(buf + L::kRowLoads * 1024);
    i32x8 fw[TW][2];
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint8_t *r = buf + (BM + (wt0 + tw) * 32) * 128;
        fw[tw][ks] = mm_lds(r + off0[ks], r + off1[ks]);
      }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const uint8_t *r = buf + (at0 + tt) * 32 * 128;
      const i32x8 fa0 = mm_lds(r + off0[0], r + off1[0]), fa1 = mm_lds(r + off0[1], r + off1[1]);
      const float xv = xsc[(at0 + tt) * 32 + rr];
#pragma unroll
      for (int tw = 0; tw < TW; ++tw) {
        f32x16 p;
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = 0.f;
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            p = mfma32_bf16(mm_bf16(fw[tw][0][2 * i], fw[tw][0][2 * i + 1]),
                            mm_bf16(fa0[2 * i], fa0[2 * i + 1]), p);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            p = mfma32_bf16(mm_bf16(fw[tw][1][2 * i], fw[tw][1][2 * i + 1]),
                            mm_bf16(fa1[2 * i], fa1[2 * i + 1]), p);
        } else {
          p = mm_mfma(fw[tw][0], fa0, p);
          p = mm_mfma(fw[tw][1], fa1, p);
        }
        const float sc = xv * __int_as_float(__builtin_amdgcn_readlane(
                                  __float_as_int(held[tw]), s % kWave));
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[tt][tw][j] = __builtin_fmaf(sc, p[j], acc[tt][tw][j]);
      }
    }
    slot = slot == NS - 1 ? 0 : slot + 1;
  }

  // register j of a 32x32 tile: weight row 8 (j / 4) + 4 rh + j % 4, row rr
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    const int m = m0 + (at0 + tt) * 32 + rr;
    if (m >= a.M) continue;
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + (wt0 + tw) * 32 + g * 8 + rh * 4;
        const size_t o = (size_t)m * a.N + n;
        const f32x16 &v = acc[tt][tw];
        if (a.N % 4 == 0) {
          if (n >= a.N) continue;
          if (F32) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.y) + o) =
                f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          } else {
            uint2 b;
            b.x = f32_to_bf16_bits(v[4 * g]) | (uint32_t)f32_to_bf16_bits(v[4 * g + 1]) << 16;
            b.y = f32_to_bf16_bits(v[4 * g + 2]) | (uint32_t)f32_to_bf16_bits(v[4 * g + 3]) << 16;
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + o) = b;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (n + e >= a.N) continue;
            if (F32)
              static_cast<float *>(a.y)[o + e] = v[4 * g + e];
            else
              static_cast<uint16_t *>(a.y)[o + e] = f32_to_bf16_bits(v[4 * g + e]);
          }
        }
      }
  }
}

template <int BM, int BN, int WM>
static hipError_t mm_launch(const MatmulArgs &a, hipStream_t stream) {
  const unsigned long long tiles =
      (((unsigned long long)a.M + BM - 1) / BM) * (((unsigned long long)a.N + BN - 1) / BN);
  if (tiles >= 1ull << 31) return hipErrorInvalidValue;  // refused ahead, by matmul_fp8_fits
  const dim3 grid((unsigned)(tiles < kMmLine ? tiles : kMmLine),
                  (unsigned)((tiles + kMmLine - 1) / kMmLine));
  if (a.f32)
    return launch(matmul_fp8_kernel<BM, BN, WM, true>, grid, dim3(kMmThreads), stream, a);
  return launch(matmul_fp8_kernel<BM, BN, WM, false>, grid, dim3(kMmThreads), stream, a);
}

hipError_t launch_matmul_fp8(const MatmulArgs &a, hipStream_t stream) {
  return mm_launch<64, 128, 2>(a, stream);
}

}  // namespace moe

// Product of E4M3 rows with E4M3 weights, a scale for each block of 128:
//
//   y[m, n] = sum over blocks b of 128 columns of
//             (xs[m, b] * ws[n / 128, b]) * sum over c in b of x[m, c] * w[n, c]
//
// A block's sum is a chain of matrix instructions from zero, folded into the fp32
// accumulator once with the product of the two scales in fp32.
//
// Codes are turned into bf16, which holds every one of them, and go through the
// 32x32x16 bf16 instruction: products are exact and sums fp32's, whatever the result's
// type.  The 8-bit instructions (both the 32x32x64 and the 32x32x16 one) align the
// products of eight neighbouring columns to the largest of the eight and drop what
// lies more than 13 bits below it, seen on MI355X with single products beside a large
// one: over random codes their sums are 1.5e-5 of the result's norm off, which a
// bf16 result's own rounding of 1.7e-3 hides, but where two large products cancel the
// small ones beside them are lost.  A caller who can bear that asks for short sums
// (bf16 results only) and gets the 8-bit 32x32x64 one, twice as fast for many rows.
//
// A workgroup computes BM rows by BN weight rows.  A stage of its LDS ring
// (ring.h) is one block of 128 columns: a 128-byte line of each row, and the
// rows' scales for that block.
//
// Where tiles are many, bound by matrix and vector instructions, which take turns: 8192
// rows by 4096 x 4096 take 250 us in bf16 and 248 in fp32, calls one after another; of
// 529 thousand cycles the matrix unit is busy 262 and the vector instructions, half of
// them conversions of codes, take 242.  With short sums 131 us; 131 and 106 of 281
// thousand cycles (the products alone, without loads, 98 us).  Bound by what a stage
// waits for where tiles are few: 777 rows by 1416 x 1152 take 9.7 us in a trace, their
// bytes 1.1 (MI355X).
#include <type_traits>

#include "e4m3.h"
#include "kernels.h"
#include "ring.h"

namespace moe {

constexpr int kMmLds = 160 * 1024;
// Workgroups in x: a grid takes fewer than 2^32 threads in each dimension.
constexpr unsigned kMmLine = 1u << 22;
constexpr unsigned kMmGroup = 8;  // tiles of rows that share a tile of weights on an XCD
constexpr int kMmPanel = 8;  // stages whose row scales are loaded together

// 32x32x64 E4M3 x E4M3; constant zero scales select the form that takes none.
__device__ __forceinline__ f32x16 mm_mfma(const i32x8 &a, const i32x8 &b, const f32x16 &c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ i32x8 mm_lds(const uint8_t *p0, const uint8_t *p1) {
  const i32x4 lo = *reinterpret_cast<const i32x4 *>(p0);
  const i32x4 hi = *reinterpret_cast<const i32x4 *>(p1);
  return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// Barrier of the ring (ring.h) behind this wave's LDS reads: what they read may be
// overwritten once every wave is here.
__device__ __forceinline__ void mm_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Where in a panel of scales row r has that of stage s: 32 rows of one stage lie in
// 32 banks.
__device__ __forceinline__ int panel_at(int r, int s) { return r * 8 + (s ^ ((r >> 3) & 7)); }

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

// WM x WN waves, each TT x TW tiles of 32 x 32, and KS such groups of waves, which
// take every KS-th block of columns; PER workgroups to a compute unit.
// LDS: panels of row scales [group][2][BM][kMmPanel], then the ring.
template <int BM, int BN, int WM, int WN, int KS, int PER>
struct MmTile {
  static constexpr int kWaves = WM * WN, kThreads = KS * kWaves * kWave;
  static constexpr int kTT = BM / 32 / WM, kTW = BN / 32 / WN;
  static_assert(kTT * WM * 32 == BM && kTW * WN * 32 == BN, "whole tiles to every wave");
  // loads of a wave in a stage, 8 rows each, and in a panel, 8 rows each
  static constexpr int kJA = BM / 8 / kWaves, kJW = BN / 8 / kWaves;
  static_assert(kJA * kWaves * 8 == BM && kJW * kWaves * 8 == BN, "the same loads to every wave");
  static_assert(kJA < kMmPanel, "a panel is under way before its first stage is");
  static constexpr int kPanels = 2 * BM * kMmPanel * 4;  // of a group
  static constexpr int kBlock = (BM + BN) * 128;         // of a group in a stage
  static constexpr int kSlot = KS * kBlock;
  static constexpr int kFit = (kMmLds / PER - KS * kPanels) / kSlot;
  static constexpr int kDepth = kFit < kMmPanel - kJA + 1 ? kFit : kMmPanel - kJA + 1;
  static_assert(kDepth >= 2, "one stage loads while one is read");
};

// MODE: what the kernel does with its sums (dense_rule.h).
template <int BM, int BN, int WM, int WN, int KS, int PER, int MODE>
__global__ __launch_bounds__(KS *WM *WN *kWave, PER *KS *WM *WN / 4) void matmul_fp8_kernel(
    MatmulArgs a) {
  using L = MmTile<BM, BN, WM, WN, KS, PER>;
  constexpr int TT = L::kTT, TW = L::kTW, NS = L::kDepth, SLOT = L::kSlot, NW = L::kWaves;
  constexpr int JA = L::kJA, JW = L::kJW;
  constexpr bool WIDE = MODE != kMmShort, GATEUP = mm_gateup(MODE);
  constexpr int BF = GATEUP ? BN / 2 : BN;  // columns of y
  static_assert(!GATEUP || 128 % BF == 0, "a tile's gate (up) rows lie in one block of scales");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KS * L::kPanels + NS * SLOT];
  uint8_t *const ring = lds + KS * L::kPanels;
  const uint32_t lds_at = lds_addr(lds);
  const int lane = lane_id();
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = all / NW, wv = all % NW;
  const unsigned tiles_n = ((unsigned)a.N + BF - 1) / BF;
  // Workgroups go to the eight XCDs in turn.  Each XCD takes a run of the tiles, in
  // an order that leaves the first kMmGroup tiles of rows for the next of weights:
  // what runs on it at a time shares few rows and weights, and its L2 holds them.
  const unsigned tiles_m = ((unsigned)a.M + BM - 1) / BM, tiles = tiles_m * tiles_n;
  const unsigned block = blockIdx.y * kMmLine + blockIdx.x;
  if (block >= tiles) return;  // the last line of workgroups may end past the tiles
  const unsigned xcd = block % 8, at = xcd * (tiles / 8) + min(xcd, tiles % 8) + block / 8;
  const unsigned strip = at / (kMmGroup * tiles_n);  // kMmGroup tiles of rows, all of weights
  const unsigned high = min((unsigned)kMmGroup, tiles_m - strip * kMmGroup);
  const unsigned in = at - strip * kMmGroup * tiles_n;
  const int m0 = (int)(strip * kMmGroup + in % high) * BM, n0 = (int)(in / high) * BF;
  // stage s of this group is block s KS + group of the columns; past the last block
  // a group loads the last again and leaves it
  const int K = a.K, blocks = K / 128, nst = (blocks + KS - 1) / KS;
  auto block_of = [&](int s) { return min(s * KS + group, blocks - 1); };

  // load i of rows (weights) fills stage rows 8 i .. 8 i + 7, a lane 16 bytes of one
  // (rows past the last read the last); load i of a panel the scales of these rows
  // for eight stages
  const int lr = lane >> 3;
  const uint8_t *xb = a.x + (size_t)m0 * K, *wb = a.w + (size_t)n0 * K;
  const uint8_t *wb1 = GATEUP ? a.w1 + (size_t)n0 * K : nullptr;
  const float *sb = a.xs + (size_t)m0 * blocks;
  uint32_t xoff[JA], woff[JW];
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    const int r = (wv + NW * j) * 8 + lr, row = min(r, a.M - 1 - m0);
    xoff[j] = (uint32_t)row * (uint32_t)K + ring_slot(r, lane & 7) * 16;
  }
#pragma unroll
  for (int j = 0; j < JW; ++j) {
    const int r = (wv + NW * j) * 8 + lr;
    // gate and up alternate in groups of 16 rows
    const int row = GATEUP ? (r >> 5) * 16 + (r & 15) : r;
    woff[j] = (uint32_t)min(row, a.N - 1 - n0) * (uint32_t)K + ring_slot(BM + r, lane & 7) * 16;
  }
  // (formed from an opaque lane number where it is used, once in eight stages: kept
  // for the whole loop it would be the registers that the largest tiles lack)
  auto issue_scales = [&](int panel, int j) {
    int l = lane;
    asm volatile("" : "+v"(l));
    const int load = wv + NW * j, st = (l & 7) ^ (load & 7);  // see panel_at
    const int row = min(load * 8 + (l >> 3), a.M - 1 - m0);
    const uint32_t off = (uint32_t)(row * blocks + block_of(panel * kMmPanel + st)) * 4u;
    mm_dma4(off, sb, lds_at + (uint32_t)(group * L::kPanels + (panel & 1) * BM * kMmPanel * 4 +
                                         load * 256));
  };
  const uint32_t group_at = lds_at + (uint32_t)(KS * L::kPanels + group * L::kBlock);
  auto issue_x = [&](int s, int slot, int j) {
    mm_dma16(xoff[j], xb + (size_t)block_of(s) * 128,
             group_at + (uint32_t)(slot * SLOT + (wv + NW * j) * 1024));
  };
  auto issue_w = [&](int s, int slot, int j) {
    const uint8_t *from = GATEUP && ((wv + NW * j) >> 1 & 1) ? wb1 : wb;
    mm_dma16(woff[j], from + (size_t)block_of(s) * 128,
             group_at + (uint32_t)(slot * SLOT + BM * 128 + (wv + NW * j) * 1024));
  };

  // this wave's tiles, and the scales of its weight rows' blocks: those of 64
  // stages are held by the lanes.  The empty asm takes them as an operand, so that
  // the wait for them stands here; where they are used, stage by stage, it would
  // wait for every load in flight, the ring's included.
  const int at0 = wv / WN * TT, wt0 = wv % WN * TW;
  constexpr int NH = GATEUP ? 2 : TW;  // gate, up; or one for each tile of the wave
  float held[NH];
  auto hold = [&](int s) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const float *from = GATEUP && i == 1 ? a.ws1 : a.ws;
      const int row = GATEUP ? n0 : min(n0 + (wt0 + i) * 32, a.N - 1);
      held[i] = from[(size_t)(row / 128) * blocks + block_of(s + lane)];
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) asm volatile("" : "+v"(held[i]));
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
  for (int j = 0; j < JA; ++j) issue_scales(0, j);
#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nst) {
#pragma unroll
      for (int j = 0; j < JA; ++j) issue_x(s, s, j);
#pragma unroll
      for (int j = 0; j < JW; ++j) issue_w(s, s, j);
    }
  int slot = 0;
  auto stage = [&](int s, auto more) {
    constexpr bool MORE = decltype(more)::value;  // stage s + NS - 1 is loaded meanwhile
    if (s != 0 && s % kWave == 0) hold(s);
    // the loads of later stages stay under way; a panel's, of which there may be
    // more, only make the wait longer
    if (MORE || s + NS - 2 < nst)
      wait_vm_imm<(NS - 2) * (JA + JW)>();
    else
      wait_vm_imm<0>();
    mm_barrier();  // stage s is in LDS for everyone; stage s - 1 is consumed
    const int ahead = s + NS - 1, to = slot == 0 ? NS - 1 : slot - 1;
    const int panel = s / kMmPanel;
    if (s % kMmPanel < JA && (panel + 1) * kMmPanel < nst) issue_scales(panel + 1, s % kMmPanel);
    const uint8_t *buf = ring + slot * SLOT + group * L::kBlock;
    const float *xsc = reinterpret_cast<const float *>(lds + group * L::kPanels) +
                       (panel & 1) * BM * kMmPanel;
    slot = slot == NS - 1 ? 0 : slot + 1;
    if (KS > 1 && s * KS + group >= blocks) return;  // in the last stage: nothing is under way
    i32x8 fw[TW][2];
    float wsc[NH];
#pragma unroll
    for (int i = 0; i < NH; ++i)
      wsc[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(held[i]), s % kWave));
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint8_t *r = buf + (BM + (wt0 + tw) * 32) * 128;
        fw[tw][ks] = mm_lds(r + off0[ks], r + off1[ks]);
      }
    bf16x8 bw[TW][8];  // the same in bf16, for the bf16 instruction
    if constexpr (WIDE) {
#pragma unroll
      for (int tw = 0; tw < TW; ++tw)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          bw[tw][i] = e4m3_bf16x8(fw[tw][i / 4][2 * (i % 4)], fw[tw][i / 4][2 * (i % 4) + 1]);
    }
    // Tile by tile: its products, behind them the previous tile's sums into the
    // accumulators (which the matrix unit then covers) and some loads of a later stage.
    f32x16 p[2];
    float xv[TT];
    auto fold = [&](int t) {
      // of gate and up: rows 0-15 of a tile are gate's, registers 0-7
      const int tt = t / TW, tw = t % TW;
      const float sc = xv[tt] * wsc[GATEUP ? 0 : tw], sc1 = GATEUP ? xv[tt] * wsc[NH - 1] : sc;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        acc[tt][tw][j] = __builtin_fmaf(j < 8 ? sc : sc1, p[t & 1][j], acc[tt][tw][j]);
    };
    i32x8 fa[2];
    bf16x8 ba[8];
#pragma unroll
    for (int t = 0; t < TT * TW; ++t) {
      const int tt = t / TW, tw = t % TW;
      if (tw == 0) {
        const uint8_t *r = buf + (at0 + tt) * 32 * 128;
        fa[0] = mm_lds(r + off0[0], r + off1[0]);
        fa[1] = mm_lds(r + off0[1], r + off1[1]);
        xv[tt] = xsc[panel_at((at0 + tt) * 32 + rr, s % kMmPanel)];
        if constexpr (WIDE) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            ba[i] = e4m3_bf16x8(fa[i / 4][2 * (i % 4)], fa[i / 4][2 * (i % 4) + 1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) p[t & 1][j] = 0.f;
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[t & 1] = mfma32_bf16(bw[tw][i], ba[i], p[t & 1]);
      } else {
        p[t & 1] = mm_mfma(fw[tw][0], fa[0], p[t & 1]);
        p[t & 1] = mm_mfma(fw[tw][1], fa[1], p[t & 1]);
      }
      if (t > 0) fold(t - 1);
      constexpr int JP = (JA + JW + TT * TW - 1) / (TT * TW), JL = JP < 2 ? 2 : JP;
      if constexpr (MORE) {
#pragma unroll
        for (int j = t * JL; j < (t + 1) * JL; ++j) {
          if (j < JW) issue_w(ahead, to, j);
          else if (j < JA + JW) issue_x(ahead, to, j - JW);
        }
      }
    }
    fold(TT * TW - 1);
  };
  int s = 0;
  for (; s + NS - 1 < nst; ++s) stage(s, std::true_type{});
  for (; s < nst; ++s) stage(s, std::false_type{});
  if constexpr (KS > 1) {
    // the groups' sums, added in the order of the groups
    constexpr int kTile = TT * TW * 16 * kWave;
    static_assert((KS - 1) * NW * kTile * 4 <= KS * L::kPanels + NS * SLOT, "room for the sums");
    float *const sums = reinterpret_cast<float *>(lds);
    mm_barrier();  // every wave is done with the ring (no load is under way)
    if (group != 0) {
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int tw = 0; tw < TW; ++tw)
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<f32x4 *>(sums + ((group - 1) * NW + wv) * kTile +
                                       (((tt * TW + tw) * 4 + j / 4) * kWave + lane) * 4) =
                f32x4{acc[tt][tw][j], acc[tt][tw][j + 1], acc[tt][tw][j + 2], acc[tt][tw][j + 3]};
    }
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 1; g < KS; ++g)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int tw = 0; tw < TW; ++tw)
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(
                sums + ((g - 1) * NW + wv) * kTile +
                (((tt * TW + tw) * 4 + j / 4) * kWave + lane) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[tt][tw][j + e] += v[e];
          }
  }

  constexpr int kSums = (KS - 1) * BM * BN * 4;
  constexpr int kLds = KS * L::kPanels + NS * SLOT;
  if constexpr (GATEUP) {
    // h takes the place of registers 0-7: features 8 (j / 4) + 4 rh + j % 4 of 16
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int tw = 0; tw < TW; ++tw)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[tt][tw][j] = swiglu(acc[tt][tw][j], acc[tt][tw][8 + j]);
  }
  if constexpr (MODE == kMmSwigluCodes) {
    // A row's block of 128 features is spread over the WN waves of its rows: they
    // exchange maxima, then put the codes together so that stores are whole lines.
    static_assert(BF == 128, "a tile holds whole blocks");
    constexpr int LINE = 128 + 16;
    static_assert(kSums + BM * WN * 4 + BM * LINE <= kLds, "room for maxima and codes");
    float *const tops = reinterpret_cast<float *>(lds + kSums);
    uint8_t *const codes = lds + kSums + BM * WN * 4;
    if (KS == 1) mm_barrier();  // every wave is done with the ring (no load is under way)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      float top = 0.f;
#pragma unroll
      for (int tw = 0; tw < TW; ++tw)
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(acc[tt][tw][j]));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (rh == 0) tops[((at0 + tt) * 32 + rr) * WN + wv % WN] = top;
    }
    __syncthreads();
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int row = (at0 + tt) * 32 + rr;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < WN; ++i) top = fmaxf(top, tops[row * WN + i]);
      // (maxima leave NaN out: where top is 0 the block may hold NaN, which gets a NaN's
      // code under the scale 1 as zeros get zeros')
      const float sc = qb_scale(top);
      bool exact;
      const float rcp = quant_rcp(sc, &exact);
#pragma unroll
      for (int tw = 0; tw < TW; ++tw)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f32x16 &v = acc[tt][tw];
          const float four[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          *reinterpret_cast<uint32_t *>(codes + row * LINE + (wt0 + tw) * 16 + g * 8 + rh * 4) =
              quant_e4m3_x4(four, sc, rcp, exact, false);
        }
      if (wv % WN == 0 && rh == 0 && m0 + row < a.M)
        a.hs[(size_t)(m0 + row) * (a.N / 128) + n0 / 128] = sc;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BM / 8 / NW; ++i) {
      const int row = (i * NW + wv) * 8 + lr;
      if (m0 + row < a.M)
        *reinterpret_cast<i32x4 *>(a.hq + (size_t)(m0 + row) * a.N + n0 + (lane & 7) * 16) =
            *reinterpret_cast<const i32x4 *>(codes + row * LINE + (lane & 7) * 16);
    }
    return;
  }

  // Register j of a 32x32 tile: weight row 8 (j / 4) + 4 rh + j % 4, row rr.  A wave
  // turns its tiles in LDS, 32 rows at a time, so that its stores are whole lines;
  // rows of y that do not start at multiples of 16 bytes are stored as they lie.
  constexpr int ES = MODE == kMmBf16 || MODE == kMmShort ? 2 : 4;
  constexpr int TF = GATEUP ? 16 : 32;    // columns of a tile
  constexpr int CH = TW * TF * ES / 16;   // 16-byte chunks of a row
  constexpr int LINE = CH * 16 + 16;      // of a row in LDS
  constexpr int RPI = kWave / CH < 32 ? kWave / CH : 32;  // rows of a store
  // (behind the groups' sums, which another wave may still be reading)
  static_assert(kSums + NW * 32 * LINE <= kLds, "every wave has room");
  const int nw = n0 + wt0 * TF;  // first column of this wave
  if ((long long)a.N * ES % 16 == 0) {
    if (KS == 1) mm_barrier();  // every wave is done with the ring (no load is under way)
    uint8_t *const mine = lds + kSums + wv * 32 * LINE;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
#pragma unroll
      for (int tw = 0; tw < TW; ++tw)
#pragma unroll
        for (int g = 0; g < TF / 8; ++g) {
          const f32x16 &v = acc[tt][tw];
          uint8_t *to = mine + rr * LINE + (tw * TF + g * 8 + rh * 4) * ES;
          if (ES == 4) {
            *reinterpret_cast<f32x4 *>(to) =
                f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
          } else {
            uint2 b;
            b.x = f32_to_bf16_bits(v[4 * g]) | (uint32_t)f32_to_bf16_bits(v[4 * g + 1]) << 16;
            b.y = f32_to_bf16_bits(v[4 * g + 2]) | (uint32_t)f32_to_bf16_bits(v[4 * g + 3]) << 16;
            *reinterpret_cast<uint2 *>(to) = b;
          }
        }
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int r = i * RPI + lane / CH, c = lane % CH;
        const int m = m0 + (at0 + tt) * 32 + r, n = nw + c * (16 / ES);
        const i32x4 v = *reinterpret_cast<const i32x4 *>(mine + r * LINE + c * 16);
        if (lane < RPI * CH && m < a.M && n < a.N)
          *reinterpret_cast<i32x4 *>(static_cast<uint8_t *>(a.y) + ((size_t)m * a.N + n) * ES) = v;
      }
    }
    return;
  }
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    const int m = m0 + (at0 + tt) * 32 + rr;
    if (m >= a.M) continue;
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int j = 0; j < TF / 2; ++j) {
        const int n = nw + tw * TF + j / 4 * 8 + rh * 4 + j % 4;
        if (n >= a.N) continue;
        const size_t o = (size_t)m * a.N + n;
        if (ES == 4)
          static_cast<float *>(a.y)[o] = acc[tt][tw][j];
        else
          static_cast<uint16_t *>(a.y)[o] = f32_to_bf16_bits(acc[tt][tw][j]);
      }
  }
}

template <int MODE, int BM, int BN, int WM, int WN, int KS, int PER>
static hipError_t mm_launch(const MatmulArgs &a, hipStream_t stream) {
  constexpr int BF = mm_gateup(MODE) ? BN / 2 : BN;
  const unsigned long long tiles =
      (((unsigned long long)a.M + BM - 1) / BM) * (((unsigned long long)a.N + BF - 1) / BF);
  const dim3 grid((unsigned)(tiles < kMmLine ? tiles : kMmLine),
                  (unsigned)((tiles + kMmLine - 1) / kMmLine));
  return launch(matmul_fp8_kernel<BM, BN, WM, WN, KS, PER, MODE>, grid,
                dim3(KS * WM * WN * kWave), stream, a);
}

hipError_t launch_gateup_fp8(const MatmulArgs &a, hipStream_t stream) {
  double t;
  if (a.hq) switch (mm_best(kMmSwigluCodes, a.M, a.N, a.K, &t)) {
      case k64x256: return mm_launch<kMmSwigluCodes, 64, 256, 2, 4, 1, 1>(a, stream);
      default: return mm_launch<kMmSwigluCodes, 128, 256, 2, 4, 1, 1>(a, stream);
    }
  switch (mm_best(kMmSwiglu, a.M, a.N, a.K, &t)) {
    case k32x64: return mm_launch<kMmSwiglu, 32, 64, 1, 2, 4, 1>(a, stream);
    case k64x64: return mm_launch<kMmSwiglu, 64, 64, 2, 2, 2, 1>(a, stream);
    default: return mm_launch<kMmSwiglu, 64, 128, 2, 2, 2, 1>(a, stream);
  }
}

template <int MODE>
static hipError_t mm_product(const MatmulArgs &a, hipStream_t stream) {
  double t;
  switch (mm_best(MODE, a.M, a.N, a.K, &t)) {
    case k32x32: return mm_launch<MODE, 32, 32, 1, 1, 8, 1>(a, stream);
    case k32x64: return mm_launch<MODE, 32, 64, 1, 2, 4, 1>(a, stream);
    case k64x64: return mm_launch<MODE, 64, 64, 2, 2, 2, 1>(a, stream);
    case k64x128: return mm_launch<MODE, 64, 128, 2, 2, 2, 1>(a, stream);
    case k64x128Two: return mm_launch<MODE, 64, 128, 2, 2, 1, 2>(a, stream);
    case k128x256: return mm_launch<MODE, 128, 256, 2, 4, 1, 1>(a, stream);
    default:
      if constexpr (MODE == kMmShort) return mm_launch<MODE, 256, 256, 2, 4, 1, 1>(a, stream);
      return hipErrorInvalidValue;  // mm_best names no other tiles for the others
  }
}

hipError_t launch_matmul_fp8(const MatmulArgs &a, hipStream_t stream) {
  if (a.f32) return mm_product<kMmF32>(a, stream);
  return a.short_sums ? mm_product<kMmShort>(a, stream) : mm_product<kMmBf16>(a, stream);
}

}  // namespace moe

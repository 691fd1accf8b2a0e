// Persistent grouped GEMM for the routed-MoE FFN with MXFP4 weights (mx4.h)
// and bf16 activations: one kernel per projection, fp32 accumulation.
//
//   gate/up: h[i, n] = bf16(silu(g) u),  g = sum_c Wg[e, n, c] x[t, c],  u likewise with Wu
//   down:    y[i, n] = sum_c Wd[e, n, c] h[i, c]
//
// for sorted row i of expert e and token t; h is rounded to bf16 because it is
// the second product's operand in the matrix unit, as in the bf16 kernels, and
// nothing else is rounded to fewer than 32 bits.  (That costs accuracy: outputs
// in bf16 are 0.0023 to 0.0024 of their norm from the formulas instead of
// 0.0017.  A second bf16 part, as the single-token kernels have it, would
// double the products of down, which is what bounds it from about 48 rows an
// expert on, and its activation rows, which decide the tile classes below
// that.)  Weights stay codes until the
// products: a lane reads 16 bytes of a weight row, 32 codes, exactly one scale
// group, and converts them in registers, so no pass over expanded weights
// exists and a weight costs 4.25 bits of memory traffic.  The order of a
// reduction follows from that (MFMA j of a step multiplies columns
// 8 j .. 8 j + 7 of each lane group's scale group); it is fixed for a tile
// height, and tile heights depend on the routing alone.
//
// What bounds an expert's tile goes with its rows, so there are three ways
// through it (times: 256 experts, d 4096, f 2048, gate/up; MI355X):
//   up to 16 rows   m4_direct  the weight stream: 401 tokens of top-6, about nine rows
//                              an expert, 413 us = 5.5 TB/s of codes and scales
//   17 to 64 rows   m4_stream  the stream, and from about 48 rows the matrix unit as much:
//                              24 rows an expert 520 us, 48 rows 605, 64 rows 690
//   more, and what the  m4_item    the matrix unit: 180 rows 1.53 ms, 256 rows 1.96 ms
//   others do not take             = 1.12 PFLOP/s, where the library's dense bf16 product
//                                  reaches 1.1 to 1.3 on this card
// The tile list, the queues that hand tiles out (M4Queues) and the rules for
// tile heights (mx4_schedule_kernel) are further down.
#include "kernels.h"
#include "mx4.h"
#include "ring.h"

namespace moe {

constexpr int kM4Queues = 8;

// Heads of a projection's work queues, and the workgroups that have left.
struct M4Heads {
  unsigned long long head[kM4Queues];
  int left, pad;
};

// What the plan leaves at the start of the workspace.
struct M4Schedule {
  int n_tiles;  // entries of the tile list, tallest capacity first
  int n_small;  // tiles of at most kM4DirectRows rows, the last n_small entries
  int n_stream;  // tiles for m4_stream ahead of them
  int many;      // whether items of tiles of few rows have twice the weight rows
  M4Heads heads[2];  // gate/up, down
};
static_assert(sizeof(M4Schedule) <= sizeof(Schedule), "has the schedule's place");

struct Mx4Args {
  const uint16_t *act;           // gate/up: x [T, K]; down: h [R, K]
  const int32_t *sorted_routes;  // gate/up: token of sorted row i is sorted_routes[i] / k
  int k;
  const uint8_t *w0, *w1;  // codes [E, N, K / 2]: gate (or down), up
  const uint8_t *s0, *s1;  // scales [E, N, K / 32] of w0, w1
  void *out;               // gate/up: h bf16 [R, N]; down: y fp32 [R, N]
  int N, K;
  const Tile *tiles;
  const M4Schedule *sch;
  M4Heads *heads;      // of the work queues (M4Queues), zeroed by the plan
};

constexpr int kM4Threads = 512;
constexpr int kM4Waves = kM4Threads / kWave;
constexpr int kM4Lds = 160 * 1024;  // the whole LDS of a workgroup
constexpr int kM4Ring = kM4Lds - 64;  // what the items use of it
constexpr int kM4WRows = 256;        // weight rows per item of the ring

// How an item of 256 weight rows and AR activation rows is laid out.
//
// Activations come in stages of KB 64-column blocks (a 128-byte line of each
// row per block), NS slots; codes in groups of GB blocks (16 GB bytes of each
// weight row), NB buffers.  Whole 128-byte lines of codes (GB = 4) matter:
// with 32-byte pieces in step with 64-column stages the requests of the codes
// alone, one per row and piece, were more than those of the activations
// (MI355X, 8192 tokens: gate/up without its products 1.10 ms).  Scales: 16 bytes per row for 8 blocks, two buffers.
//
// Split: tiles of up to 64 rows.  Wave w takes weight tiles 2 (w % 4) and
// 2 (w % 4) + 1, every activation tile, and block w / 4 of each stage's two;
// the two halves of the sums meet in LDS at the end.  Each weight is decoded
// once and each activation tile read serves two products.  Taller tiles:
// wave w takes the same weight tiles and half w / 4 of the activation tiles.
template <int AR>
struct M4Layout {
  static constexpr bool kSplit = AR <= 64;
  static constexpr int KB = kSplit ? 2 : 1;
  static constexpr int GB = AR == 256 ? 2 : 4;
  static constexpr int NB = kSplit || AR == 256 ? 3 : 2;
  static constexpr int S = GB / KB;  // stages per group of codes
  static constexpr int TT = kSplit ? AR / 32 : AR / 64;
  static constexpr int TW = 2;
  static constexpr int kAct = AR * 128 * KB;
  static constexpr int kCodes = kM4WRows * 16 * 2 * GB;
  static constexpr int kScales = kM4WRows * 16;
  static constexpr int kFit = (kM4Ring - NB * kCodes - 2 * kScales) / kAct;
  // A group's codes go out NB - 1 groups ahead, after the activations of that
  // stage; with no more slots than this they are older than the activations
  // of the group's first stage, which alone then decide what a stage waits for.
  static constexpr int kMost = (NB - 1) * S;
  static constexpr int NS = kFit < kMost ? kFit : kMost;
  static constexpr int kCodeBase = NS * kAct;
  static constexpr int kScaleBase = kCodeBase + NB * kCodes;
  static_assert(NS >= 2 && kScaleBase + 2 * kScales <= kM4Ring, "fits");
  static_assert(!kSplit || 4 * TW * TT * 4096 <= kM4Ring, "the sums fit");
  __device__ static int atile(int wv, int tt) { return kSplit ? tt : (wv >> 2) * TT + tt; }
  __device__ static int wtile(int wv, int tw) { return (wv & 3) * 2 + tw; }
};

// 16-byte chunk c of the codes of weight row r is stored at this slot of the
// row's 2 GB: 16 lanes reading one chunk of 16 consecutive rows then touch
// 16 distinct 16-byte slots of a 256-byte window.
template <int GB>
__device__ __forceinline__ int m4_slot(int r, int c) {
  return c ^ ((r / (8 / GB)) & (2 * GB - 1));
}

// Direct global->LDS load of 4 bytes per lane to LDS byte address
// lds_byte_addr + 4 * lane (see dma16).
__device__ __forceinline__ void dma4(const void *src, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(lds_byte_addr)
               : "memory");
}

// The loads of ring.h from a uniform base plus a 32-bit offset per lane.
__device__ __forceinline__ void m4_dma16(const void *base, uint32_t off, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_byte_addr)
               : "memory");
}
__device__ __forceinline__ void m4_dma16_nt(const void *base, uint32_t off, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
               :
               : "v"(off), "s"(base), "s"(lds_byte_addr)
               : "memory");
}

__device__ __forceinline__ f32x4 m4_quad(const f32x16 &v, int g) {
  return f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
}

// How many of the n stages before stage i of a group of S are first in theirs.
__host__ __device__ constexpr int m4_firsts(int i, int n, int S) {
  int c = 0;
  for (int u = 1; u <= n; ++u) c += (i - u + 64 * S) % S == 0 ? 1 : 0;
  return c;
}

// The steady wait of stage i of a group (below); i is a constant once unrolled.
template <int JA, int JW, int NS, int S>
__device__ __forceinline__ void m4_wait(int i) {
  const int firsts = m4_firsts(i, NS - 1, S);
  if (firsts == 0)
    wait_vm_imm<JA *(NS - 2)>();
  else if (firsts == 1)
    wait_vm_imm<JA *(NS - 2) + JW>();
  else
    wait_vm_imm<JA *(NS - 2) + 2 * JW>();
}

template <int N>
struct M4Tiles {
  static constexpr int n = N;
};

// 256 weight rows (features from n0) of a tile of up to AR rows.
template <bool GATEUP, int AR>
__device__ __forceinline__ void m4_item(const Mx4Args &a, const Tile &t, int n0, uint8_t *ring,
                                        uint32_t ring_lds) {
  using L = M4Layout<AR>;
  constexpr int KB = L::KB, GB = L::GB, NB = L::NB, S = L::S, NS = L::NS;
  constexpr int TT = L::TT, TW = L::TW;
  constexpr int JA = KB * AR / 8 / kM4Waves;       // activation loads (8 rows) of a wave per stage
  constexpr int JW = kM4WRows * GB / 32 / kM4Waves;  // code loads (1 KB) of a wave per group
  const int lane = vreg(lane_id());
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int K = a.K;
  const int nst = K / (64 * KB);
  const int ngr = (K / 64 + GB - 1) / GB;
  const bool half = GB == 4 && (K & 128) != 0;  // the last group has two blocks only
  // the codes of an expert's only tile are read once: past the caches, in whole lines
  const bool nt = L::kSplit && (t.ablk & kTileStream);

  // Weight row wr of the item: a row of the first or second matrix (gate/up:
  // 16-row groups alternate), counted from feature n0.
  auto wmat = [&](int wr) { return GATEUP ? (wr >> 4) & 1 : 0; };
  auto wrow = [&](int wr) {
    return GATEUP ? (wr >> 5) * 16 + (wr & 15) : min(wr, a.N - 1 - n0);
  };
  const size_t first = (size_t)t.e * a.N + n0;
  const uint8_t *const s0 = a.s0 + first * (K / 32), *const s1 = GATEUP ? a.s1 + first * (K / 32) : s0;
  // this lane's source of each of its loads in the first stage and group
  const uint8_t *act[JA];
  uint32_t codes[JW];
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    const int i = wv + kM4Waves * j;
    const int kb = i / (AR / 8);
    const int r = (i - kb * (AR / 8)) * 8 + (lane >> 3);
    const int row = t.row0 + min(r, t.nrows - 1);
    const size_t s = GATEUP ? (size_t)(a.sorted_routes[row] / vreg(a.k)) : (size_t)row;
    act[j] = reinterpret_cast<const uint8_t *>(a.act + s * K) + kb * 128 +
             ring_slot(r, lane & 7) * 16;
  }
  constexpr int LPR = 2 * GB;  // lanes per row of codes; the rows of a load are of one matrix
  constexpr int RPL = 64 / LPR;
  // all code loads of a wave are of the same matrix (they are 8 RPL rows apart)
  static_assert(kM4Waves * RPL % 32 == 0, "of the same matrix");
  const uint8_t *const w = (wmat(wv * RPL) ? a.w1 : a.w0) + first * (K / 2);
  int second = 0;  // bit j: load j brings columns of the group's second half
#pragma unroll
  for (int j = 0; j < JW; ++j) {
    const int r = (wv + kM4Waves * j) * RPL + lane / LPR;
    const int c = m4_slot<GB>(r, lane % LPR);
    codes[j] = (uint32_t)wrow(r) * (K / 2) + c * 16;
    second |= (c >= 4 ? 1 : 0) << j;
  }
  // Scales: where rows start on 16-byte borders, one load of 16 bytes per
  // lane and 64 rows by waves 4-7 (32 rows of each matrix for gate/up);
  // elsewhere loads of 4 bytes per lane and 16 rows.  Both leave 16 bytes per
  // row in LDS.
  const int aligned = vreg((K & 511) == 0);  // in a vector register, for want of a scalar one
  const bool wide = __builtin_amdgcn_readfirstlane(aligned);
  const int srow = wide ? max(wv - 4, 0) * 64 + lane : wv * 32 + (lane >> 2);
  const uint8_t *scales = (wmat(srow) ? s1 : s0) + (size_t)wrow(srow) * (K / 32);
  const uint8_t *scales16 = (wmat(srow + 16) ? s1 : s0) + (size_t)wrow(srow + 16) * (K / 32);

  auto issue_code = [&](int j, int g, int buf) {
    const int i = wv + kM4Waves * j;
    const uint8_t *base = w + (uint32_t)g * (32 * GB);
    uint32_t off = codes[j];
    // half a group: its first half twice (loaded, not used)
    if (GB == 4 && half && g == ngr - 1) off -= ((second >> j) & 1) * 64;
    const uint32_t to = ring_lds + (uint32_t)(L::kCodeBase + buf * L::kCodes + i * 1024);
    if (nt)
      m4_dma16_nt(base, off, to);
    else
      m4_dma16(base, off, to);
  };
  auto issue_scales = [&](int g) {
    if (g % (8 / GB) != 0) return;
    const uint32_t to = ring_lds + (uint32_t)L::kScaleBase + (uint32_t)(g / (8 / GB) & 1) * L::kScales;
    uint32_t off = (uint32_t)g * (2 * GB);
    if (__builtin_amdgcn_readfirstlane(aligned)) {
      if (wv >= 4) dma16(scales + off, to + (uint32_t)(wv - 4) * 1024u);
    } else {
      // words past the row's end are not there: the group's first instead
      off += (g * GB + (lane & 3) * 2) * 64 < K ? (lane & 3) * 4 : 0;
      dma4(scales + off, to + (uint32_t)wv * 512u);
      dma4(scales16 + off, to + (uint32_t)wv * 512u + 256u);
    }
  };
  auto issue_act = [&](int j, int s, int slot) {
    dma16(act[j] + (uint32_t)s * (128 * KB),
          ring_lds + (uint32_t)(slot * L::kAct + (wv + kM4Waves * j) * 1024));
  };

  const int rr = lane & 31, rh = lane >> 5;
  // whether the tile has rows in this wave's last activation tile
  const bool last = __builtin_amdgcn_readfirstlane(L::atile(wv, TT - 1) * 32 < t.nrows);
  f32x16 acc[TW][TT];
#pragma unroll
  for (int tw = 0; tw < TW; ++tw)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[tw][tt][j] = 0.f;

  // this wave's MFMAs of stage i of group g: activations in `slot`, codes in `buf`
  // with between(j) after the MFMAs of step j
  auto mma_stage = [&](auto tiles, int g, int i, int slot, int buf, auto between) {
    constexpr int N = decltype(tiles)::n;
    const int q = L::kSplit ? wv >> 2 : 0;  // this wave's block of the stage
    const uint8_t *ap = ring + slot * L::kAct + q * (AR * 128);
    const uint8_t *cp = ring + L::kCodeBase + buf * L::kCodes;
    // the scales' two bytes of block b = g GB + i KB + q of the row's
    const uint8_t *sp = ring + L::kScaleBase + (g / (8 / GB) & 1) * L::kScales +
                        (g * (GB / 2) & 3) * 4 + (i * KB + q) / 2 * 4;
    const int shift = 8 * rh + 16 * ((i * KB + q) & 1);
    // Activations of step j + 1 are read ahead of the products of step j
    // (8192 tokens: gate/up 1.66 -> 1.59 ms), for which the registers of
    // 256-row tiles do not suffice.
    constexpr bool AHEAD = AR < 256;
    bf16x8 fa[AHEAD ? 2 : 1][N];
    auto read_act = [&](int j) {
#pragma unroll
      for (int tt = 0; tt < N; ++tt)
        fa[AHEAD ? j & 1 : 0][tt] = *reinterpret_cast<const bf16x8 *>(
            ap + (L::atile(wv, tt) * 32 + rr) * 128 + ring_slot(rr, 4 * rh + j) * 16);
    };
    i32x4 raw[TW];
    uint32_t word[TW];
#pragma unroll
    for (int tw = 0; tw < TW; ++tw) {
      const int r = L::wtile(wv, tw) * 32 + rr;
      raw[tw] = *reinterpret_cast<const i32x4 *>(cp + r * (32 * GB) +
                                                 m4_slot<GB>(r, 2 * (i * KB + q) + rh) * 16);
      word[tw] = *reinterpret_cast<const uint32_t *>(sp + r * 16);
    }
    read_act(0);
    float scale[TW];
#pragma unroll
    for (int tw = 0; tw < TW; ++tw) scale[tw] = mx4_scale((word[tw] >> shift) & 0xffu);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (AHEAD) {
        if (j < 3) read_act(j + 1);
        __builtin_amdgcn_sched_barrier(0);
      } else if (j > 0) {
        read_act(j);
      }
#pragma unroll
      for (int tw = 0; tw < TW; ++tw) {
        const bf16x8 fw = mx4_decode8((uint32_t)raw[tw][j], scale[tw]);
#pragma unroll
        for (int tt = 0; tt < N; ++tt)
          acc[tw][tt] = mfma32_bf16(fw, fa[AHEAD ? j & 1 : 0][tt], acc[tw][tt]);
      }
      between(j);
    }
  };

  ring_barrier();  // every wave has read its item, which lies in the ring
  auto issue_group = [&](int g) {
#pragma unroll
    for (int j = 0; j < JW; ++j) issue_code(j, g, g);
    issue_scales(g);
  };
  issue_group(0);
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (s < nst) {
#pragma unroll
      for (int j = 0; j < JA; ++j) issue_act(j, s, s);
    }
  }
#pragma unroll
  for (int g = 1; g < NB - 1; ++g)
    if (g < ngr) issue_group(g);
  auto stages = [&](auto tiles) {
    int slot = 0, buf = 0;  // of the stage being multiplied
#pragma unroll 1
    for (int g = 0; g < ngr; ++g) {
      // What may stay in flight at the start of stage s: the activations of the
      // NS - 2 stages after it, and the codes that went out since its own
      // activations did (with the first stage of a group, after that stage's
      // activations).  Between the first groups and the last NB that is a
      // constant.  Scales are not counted: the wait is then one load longer.
      const bool steady = g * S >= NS - 1 && g + NB < ngr;
      const bool codes_too = g + NB - 1 < ngr;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int s = g * S + i;
        if (GB == 4 && i >= S / 2 && s >= nst) break;  // half a group
        if (steady) {
          m4_wait<JA, JW, NS, S>(i);
        } else {
          int n = JA * min(NS - 2, nst - 1 - s);
          if (s <= NS - 2) n += JW * min(NB - 2, ngr - 1);  // issued ahead of the loop
#pragma unroll
          for (int x = 1; x < NS; ++x) {
            const int h = g - (x - i + S - 1) / S;  // the group of stage s - x if that is its first
            if (x >= i && (x - i) % S == 0 && h >= 0 && h + NB - 1 < ngr) n += JW;
          }
          wait_vm(n);
        }
        ring_barrier();  // the stage is in LDS for everyone; stage s - 1 is consumed
        // the next loads go out between the products: all at once, ahead of
        // them, they kept the waves from starting
        const bool more = s + NS - 1 < nst;
        const auto between = [&](int j) {
          constexpr int N = JA + JW;
          const int to_slot = slot == 0 ? NS - 1 : slot - 1, to_buf = buf == 0 ? NB - 1 : buf - 1;
#pragma unroll
          for (int x = 0; x < N; ++x) {
            if (x * 4 / N != j) continue;
            if (x < JA) {
              if (more) issue_act(x, s + NS - 1, to_slot);
            } else if (i == 0 && codes_too) {
              issue_code(x - JA, g + NB - 1, to_buf);
              if (x == N - 1) issue_scales(g + NB - 1);
            }
          }
        };
        mma_stage(tiles, g, i, slot, buf, between);
        slot = slot == NS - 1 ? 0 : slot + 1;
      }
      buf = buf == NB - 1 ? 0 : buf + 1;
    }
  };
  if (L::kSplit || last)
    stages(M4Tiles<TT>{});
  else
    stages(M4Tiles<L::kSplit ? TT : TT - 1>{});

  if constexpr (L::kSplit) {
    f32x4 *sums = reinterpret_cast<f32x4 *>(ring) + (wv & 3) * (TW * TT * 256) + lane;
    ring_barrier();  // the ring makes room for the sums of waves 4-7
    if (wv >= 4) {
#pragma unroll
      for (int tw = 0; tw < TW; ++tw)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            sums[((tw * TT + tt) * 4 + g) * kWave] = m4_quad(acc[tw][tt], g);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    ring_barrier();
    if (wv >= 4) return;
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 v = sums[((tw * TT + tt) * 4 + g) * kWave];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[tw][tt][4 * g + i] += v[i];
        }
  }
  // register j of a 32x32 tile holds weight row 8*(j/4) + 4*rh + j%4, activation row rr
#pragma unroll
  for (int tt = 0; tt < TT; ++tt) {
    const int r = L::atile(wv, tt) * 32 + rr;
    if (r >= t.nrows) continue;
    const size_t row = (size_t)(t.row0 + r);
#pragma unroll
    for (int tw = 0; tw < TW; ++tw) {
      const int wt = L::wtile(wv, tw);
      if (GATEUP) {
        // rows 0-15 of the tile are gate features 16 wt + [0,16), rows 16-31 the same up features
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f32x4 gv = m4_quad(acc[tw][tt], g), uv = m4_quad(acc[tw][tt], g + 2);
          const int n = n0 + wt * 16 + g * 8 + rh * 4;
          uint2 v;
          v.x = (uint32_t)f32_to_bf16_bits(swiglu(gv[0], uv[0])) |
                ((uint32_t)f32_to_bf16_bits(swiglu(gv[1], uv[1])) << 16);
          v.y = (uint32_t)f32_to_bf16_bits(swiglu(gv[2], uv[2])) |
                ((uint32_t)f32_to_bf16_bits(swiglu(gv[3], uv[3])) << 16);
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + row * a.N + n) = v;
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int n = n0 + wt * 32 + g * 8 + rh * 4;
          if (n < a.N)
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + row * a.N + n) =
                m4_quad(acc[tw][tt], g);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ few rows

// A tile of at most 16 rows is a weight stream with little to multiply.  Its
// activation rows go to LDS whole, once per item, and every wave then streams
// weight rows of its own straight into registers, two chunks of kM4Steps
// steps in turn (the next one's loads in flight while one is multiplied):
// there is no barrier per stage, so no wave waits for another's loads, and
// LDS serves the activations only.  (Through the ring, whose stages all waves
// read at the same time, reads of activation tiles kept LDS busy for most of
// a stage: MI355X, 401 tokens, gate/up 508 us; this way 413.)
// Products are 16x16x32 MFMAs: a step is 128 columns, lane group c = l / 16
// holds the codes of group c of a weight row l % 16 (16 bytes), and MFMA j
// multiplies columns 8 j .. 8 j + 7 of the four groups.
constexpr int kM4Steps = 4;
constexpr int kM4DirectRows = 16;
constexpr int kM4ScaleRow = kM4Steps * 4 + 16;  // a weight row's scales of a chunk in LDS, padded
constexpr int kM4ScaleWave = 2 * 16 * kM4ScaleRow;
constexpr int kM4DirectAct = kM4Ring - kM4Waves * kM4ScaleWave;  // LDS for activation rows

// Row stride of the activation rows in LDS, padded: consecutive rows start
// in different banks.
__device__ __forceinline__ int m4_direct_stride(int K) { return 2 * K + 16; }
__device__ __forceinline__ bool m4_direct_fits(int K) {
  return kM4DirectRows * m4_direct_stride(K) <= kM4DirectAct;  // K <= 4,736
}
static_assert(kM4DirectRows * (2 * 4736 + 16) <= kM4DirectAct &&
                  kM4DirectRows * (2 * 4864 + 16) > kM4DirectAct,
              "the longest multiple of 128 that fits");

// One chunk of a wave's two weight tiles of 16 rows.
struct M4Chunk {
  i32x4 raw[kM4Steps][2];
  uint32_t sc[2];  // without WIDE: in lane group c the scales of step c
};

// The scales of a wave's two weight tiles for a whole row of up to eight
// chunks, in whole lines: lane l holds chunk l % 8 of rows l / 8 and l / 8 + 8.
struct M4Scales {
  i32x4 v[2][2];
};

// Output features [n0, n1) of a tile.
// WIDE (K a multiple of 1024): the scales come in whole lines, a chunk's 16
// bytes per row passing through LDS to the lanes that multiply; fetched with
// each chunk instead, 16 bytes of a line at a time, they cost twice their
// share of the bytes (MI355X, 401 tokens: gate/up 440 us, 390 without scales).
template <bool GATEUP, bool WIDE>
__device__ __forceinline__ void m4_direct(const Mx4Args &a, const Tile &t, int n0, int n1,
                                          uint8_t *lds) {
  constexpr int FG = GATEUP ? 16 : 32;  // features of a wave's two weight tiles
  const int lane = vreg(lane_id());
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane >> 4, row = lane & 15;
  const int K = a.K, nk = K / 128;
  const int stride = m4_direct_stride(K);
  const int chunks = (nk + kM4Steps - 1) / kM4Steps;
  const int groups = max(((n1 - n0) / FG - wv + kM4Waves - 1) / kM4Waves, 0);
  const int total = groups * chunks;
  uint8_t *sc_lds0 = lds + kM4DirectAct + wv * kM4ScaleWave;
  uint8_t *sc_lds = sc_lds0 + row * kM4ScaleRow;

  auto load = [&](M4Chunk &q, int i) {
    const int g = i / chunks, s = (i - g * chunks) * kM4Steps;
    const int n = n0 + (wv + kM4Waves * g) * FG;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const size_t r = (size_t)t.e * a.N + n + row + (GATEUP ? 0 : 16 * w);
      const uint8_t *codes = (GATEUP && w ? a.w1 : a.w0) + r * (K / 2) + c * 16;
      const uint8_t *scales = (GATEUP && w ? a.s1 : a.s0) + r * (K / 32);
      // steps past the end load the last one again
      if (!WIDE) q.sc[w] = *reinterpret_cast<const uint32_t *>(scales + min(s + c, nk - 1) * 4);
#pragma unroll
      for (int u = 0; u < kM4Steps; ++u)
        q.raw[u][w] = *reinterpret_cast<const i32x4 *>(codes + min(s + u, nk - 1) * 64);
    }
    asm volatile("" ::: "memory");  // issued here, not where they are used
  };
  auto load_scales = [&](M4Scales &q, int g) {
    const int n = n0 + (wv + kM4Waves * g) * FG;
    const int at = min(lane & 7, chunks - 1) * 16;
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const size_t r = (size_t)t.e * a.N + n + (lane >> 3) + 8 * h + (GATEUP ? 0 : 16 * w);
        q.v[w][h] = *reinterpret_cast<const i32x4 *>((GATEUP && w ? a.s1 : a.s0) + r * (K / 32) + at);
      }
    asm volatile("" ::: "memory");
  };
  f32x4 acc[2] = {};
  const uint8_t *mine = lds + min(row, t.nrows - 1) * stride + c * 64;
  M4Scales sa, sb;  // WIDE: of the group being multiplied, and of the next
  auto multiply = [&](const M4Chunk &q, int i) {
    const int g = i / chunks, ci = i - g * chunks, s = ci * kM4Steps;
    i32x4 ss[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (WIDE) {
        if ((lane & 7) == ci) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<i32x4 *>(sc_lds0 + (w * 16 + (lane >> 3) + 8 * h) * kM4ScaleRow) =
                sa.v[w][h];
        }
      } else {
        *reinterpret_cast<uint32_t *>(sc_lds + w * 16 * kM4ScaleRow + c * 4) = q.sc[w];
      }
      ss[w] = *reinterpret_cast<const i32x4 *>(sc_lds + w * 16 * kM4ScaleRow);
    }
    const int steps = min(kM4Steps, nk - s);
#pragma unroll
    for (int u = 0; u < kM4Steps; ++u) {
      if (u >= steps) break;
      bf16x8 fx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        fx[j] = *reinterpret_cast<const bf16x8 *>(mine + (s + u) * 256 + j * 16);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float scale = mx4_scale(((uint32_t)ss[w][u] >> (8 * c)) & 0xffu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[w] = mfma_bf16(mx4_decode8((uint32_t)q.raw[u][w][j], scale), fx[j], acc[w]);
      }
    }
    if (ci + 1 < chunks) return;
    // register r of lane l: weight row 4 (l / 16) + r, activation row l % 16
    if (row < t.nrows) {
      const int n = n0 + (wv + kM4Waves * g) * FG + 4 * c;
      const size_t o = (size_t)(t.row0 + row) * a.N + n;
      if (GATEUP) {
        uint2 v;
        v.x = (uint32_t)f32_to_bf16_bits(swiglu(acc[0][0], acc[1][0])) |
              ((uint32_t)f32_to_bf16_bits(swiglu(acc[0][1], acc[1][1])) << 16);
        v.y = (uint32_t)f32_to_bf16_bits(swiglu(acc[0][2], acc[1][2])) |
              ((uint32_t)f32_to_bf16_bits(swiglu(acc[0][3], acc[1][3])) << 16);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + o) = v;
      } else {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + o) = acc[0];
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + o + 16) = acc[1];
      }
    }
    acc[0] = f32x4{};
    acc[1] = f32x4{};
  };

  M4Chunk qa, qb;
  if (total > 0) {
    if (WIDE) load_scales(sa, 0);
    load(qa, 0);
  }
  ring_barrier();  // every wave has read its item, which lies where the rows go
  // wave w brings rows w and w + 8
  for (int r = wv; r < t.nrows; r += kM4Waves) {
    const int i = t.row0 + r;
    const size_t s = GATEUP ? (size_t)(a.sorted_routes[i] / vreg(a.k)) : (size_t)i;
    for (int p0 = 0; p0 < K / 8; p0 += 8 * kWave) {
      i32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        v[u] = *reinterpret_cast<const i32x4 *>(a.act + s * K +
                                                min(p0 + u * kWave + lane, K / 8 - 1) * 8);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<i32x4 *>(lds + r * stride + min(p0 + u * kWave + lane, K / 8 - 1) * 16) =
            v[u];
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  ring_barrier();
  // no load in the loops is conditional: where a path without it joined, the
  // compiler would have to wait for all of them
  if (total == 0) return;
  int i = 0;
  if (WIDE) {  // an even number of chunks per row
#pragma unroll 1
    for (int g = 0; g < groups; ++g) {
      load_scales(sb, min(g + 1, groups - 1));
#pragma unroll 1
      for (int ci = 0; ci < chunks; ci += 2, i += 2) {
        load(qb, i + 1);
        multiply(qa, i);
        load(qa, min(i + 2, total - 1));
        multiply(qb, i + 1);
      }
      sa = sb;
    }
  } else {
#pragma unroll 1
    for (; i + 2 < total; i += 2) {
      load(qb, i + 1);
      multiply(qa, i);
      load(qa, i + 2);
      multiply(qb, i + 1);
    }
    if (i + 1 < total) {
      load(qb, i + 1);
      multiply(qa, i);
      multiply(qb, i + 1);
    } else {
      multiply(qa, i);
    }
  }
}

// ------------------------------------------------------------------ up to 64 rows

// Tiles of 17 to 64 rows over a reduction of whole slices of 512 columns.
// Weights go straight into registers as in m4_direct, chunk by chunk of 256
// columns; of the activations two slices of up to 64 rows are in LDS, the next
// one on its way while one is multiplied, and the waves meet once per slice.
// Wave w takes weight rows [64 w, 64 w + 64) of the item's 512, which keeps
// the reads of activations at half of what LDS can do beside the products, and
// multiplies with as many 16-row tiles as hold rows (TM), by the 16x16x32
// instruction, whose rate on this card is 1.24 PFLOP/s where the ring's
// 32x32x16 has 2.1: the products, not the loads, are the longer part from
// about 40 rows on.  Against the ring,
// which multiplies 64 rows always and meets every 128 columns (MI355X, 256
// experts, d 4096, f 2048, gate/up): 24 rows an expert 670 -> 510 us, 48 rows
// 735 -> 605, 64 rows 720 -> 690.  At 48 rows the loads alone take 460 us and
// the products alone 590.
//
// Row r of a slice takes 1 KB of LDS, one load of a wave; its 16-byte chunk
// p lies at p ^ (r % 8), so that eight lanes reading one chunk of consecutive
// rows touch all banks once.
constexpr int kM4SliceCols = 512;
constexpr int kM4StreamRows = 64;
constexpr int kM4Slice = kM4StreamRows * kM4SliceCols * 2;
static_assert(2 * kM4Slice <= kM4Ring, "two slices fit");

__device__ __forceinline__ bool m4_stream_takes(int K) { return K % kM4SliceCols == 0; }

// One chunk of a wave's four weight tiles of 16 rows: two steps of 128 columns.
struct M4Chunk2 {
  i32x4 raw[2][4];
};

// 512 weight rows (features from n0) of a tile of up to 16 TM rows.
template <bool GATEUP, int TM>
__device__ __forceinline__ void m4_stream(const Mx4Args &a, const Tile &t, int n0, uint8_t *lds,
                                          uint32_t lds_base) {
  constexpr int FG = GATEUP ? 32 : 64;  // features of a wave's four weight tiles
  const int lane = vreg(lane_id());
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane >> 4, row = lane & 15;
  const int K = a.K, slices = K / kM4SliceCols;
  const int nw = n0 + wv * FG;
  // waves past the last feature keep the others company on its rows
  const size_t first = (size_t)t.e * a.N + min(nw, a.N - FG);
  const uint8_t *const w0 = a.w0 + first * (K / 2), *const w1 = GATEUP ? a.w1 + first * (K / 2) : w0;
  // tile w of a wave: gate/up: gate and up rows of 16 features, then of the next 16
  auto tile_row = [](int w) { return GATEUP ? (w >> 1) * 16 : w * 16; };
  constexpr int NO = GATEUP ? 2 : 4;
  uint32_t code_off[NO];
#pragma unroll
  for (int i = 0; i < NO; ++i) code_off[i] = (uint32_t)vreg(i * 16 + row) * (K / 2) + c * 16;

  auto load = [&](M4Chunk2 &q, int ch) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint8_t *base = (GATEUP && (w & 1) ? w1 : w0) + (uint32_t)ch * 128;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        q.raw[u][w] = *reinterpret_cast<const i32x4 *>(base + code_off[GATEUP ? w >> 1 : w] + u * 64);
    }
    asm volatile("" ::: "memory");  // issued here, not where they are used
  };
  // The scales of four slices: lane group c holds those of slice c, 16 bytes a row.
  auto load_scales = [&](i32x4 (&q)[4], int s) {
    const size_t at = (size_t)(w0 - a.w0) / 16;  // a byte of scales to 16 of codes
    const uint32_t off = (uint32_t)row * (K / 32) + (uint32_t)min(s + c, slices - 1) * 16;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      q[w] = *reinterpret_cast<const i32x4 *>((GATEUP && (w & 1) ? a.s1 : a.s0) + at +
                                            tile_row(w) * (K / 32) + off);
    asm volatile("" ::: "memory");
  };
  // source row of tile row wv + 8 l in lane l; rows past the last repeat it
  const int tile_at = t.row0 + min(wv + kM4Waves * (lane & 7), t.nrows - 1);
  const int src = GATEUP ? a.sorted_routes[tile_at] / vreg(a.k) : tile_at;
  const uint32_t act_off = (uint32_t)((lane ^ wv) * 16);
  // this wave's rows of slice s: wv, wv + 8, ..
  auto issue = [&](int s) {
    const uint32_t to = lds_base + (uint32_t)((s & 1) * kM4Slice + wv * 1024);
#pragma unroll
    for (int i = 0; i < 16 * TM / kM4Waves; ++i) {
      const size_t from = (size_t)__builtin_amdgcn_readlane(src, i) * K + (size_t)s * kM4SliceCols;
      m4_dma16(a.act + from, act_off, to + (uint32_t)(i * kM4Waves * 1024));
    }
  };

  f32x4 acc[4][TM] = {};
  i32x4 sa[4];  // scales of the four slices being multiplied
  const int sel = row * 4;
  // half of slice s, with between() behind its first products
  auto multiply = [&](const M4Chunk2 &q, int s, int half, auto between) {
    const uint8_t *ap = lds + (s & 1) * kM4Slice + row * 1024 + half * 512;
    bf16x8 fa[2][TM];
    auto read = [&](int x) {
#pragma unroll
      for (int m = 0; m < TM; ++m)
        fa[x & 1][m] = *reinterpret_cast<const bf16x8 *>(
            ap + m * 16384 + (x >> 2) * 256 + (((c * 4 + (x & 3)) ^ (lane & 7)) * 16));
    };
    read(0);
    float scale[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t v = (uint32_t)__builtin_amdgcn_ds_bpermute(
            sel + (s & 3) * 64, half == 0 ? sa[w][u] : sa[w][2 + u]);
        scale[u][w] = mx4_scale((v >> (8 * c)) & 0xffu);
      }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      if (x < 7) read(x + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const bf16x8 fw = mx4_decode8((uint32_t)q.raw[x >> 2][w][x & 3], scale[x >> 2][w]);
#pragma unroll
        for (int m = 0; m < TM; ++m) acc[w][m] = mfma_bf16(fw, fa[x & 1][m], acc[w][m]);
      }
      if (x == 0) between();
    }
  };

  M4Chunk2 qa, qb;
  load_scales(sa, 0);
  load(qa, 0);
  ring_barrier();  // every wave has read its item, which lies where the rows go
  issue(0);
  wait_vm_imm<0>();
  ring_barrier();
#pragma unroll 1
  for (int s4 = 0; s4 < slices; s4 += 4) {
    const int end = min(s4 + 4, slices);
#pragma unroll 1
    for (int s = s4; s < end; ++s) {
      load(qb, 2 * s + 1);
      // The other slice's place is free since the last barrier.  These loads
      // are older than the chunk that is loaded next and younger than this one,
      // so no wait for codes is longer for them.
      multiply(qa, s, 0, [&] {
        if (s + 1 < slices) issue(s + 1);
      });
      load(qa, min(2 * s + 2, 2 * slices - 1));
      multiply(qb, s, 1, [] {});
      wait_vm_imm<8>();  // all but the chunk's: slice s + 1 is here
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      ring_barrier();
    }
    load_scales(sa, s4 + 4);
  }
  if (nw >= a.N) return;
  // register r of lane l: weight row 4 (l / 16) + r, activation row l % 16
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    if (m * 16 + row >= t.nrows) continue;
    const size_t o = (size_t)(t.row0 + m * 16 + row) * a.N + nw + 4 * c;
    if (GATEUP) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 g = acc[2 * h][m], u = acc[2 * h + 1][m];
        uint2 v;
        v.x = (uint32_t)f32_to_bf16_bits(swiglu(g[0], u[0])) |
              ((uint32_t)f32_to_bf16_bits(swiglu(g[1], u[1])) << 16);
        v.y = (uint32_t)f32_to_bf16_bits(swiglu(g[2], u[2])) |
              ((uint32_t)f32_to_bf16_bits(swiglu(g[3], u[3])) << 16);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + o + 16 * h) = v;
      }
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w)
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + o + 16 * w) = acc[w][m];
    }
  }
}

// ------------------------------------------------------------------ kernel

// The tile list, one thread per expert: its full tiles of `cap` rows, then one
// remainder tile of the smallest capacity of 16, 64, 128, 192 and 256 rows
// that holds it (Tile::ablk in 32 rows, 1 for 16); all tiles of a class
// together, tallest class first, experts in order.  Inside a class a tile
// pays for its rows in steps of 16 (m4_stream) or 32 (m4_item).
//
// cap is 256 rows, which reads an expert's weights least often, unless the
// tiles then make fewer items than there are workgroups: 128 or 64 rows give
// more of them, each with less to multiply (777 tokens, three routes each
// over 24 experts, d 1152, f 640: gate/up 32.5 -> 18.7 us, down 23.9 -> 13.4 us).
// Tiles of up to 64 rows come in items of twice the weight rows, and those of
// 17 to 64 through m4_stream, where single items would take the workgroups
// more than one round (the same layer with E experts of 48 rows, d 4096,
// f 2048, gate/up: 16 experts, one round, 46 us single and 58 double; 24
// experts 93 and 66; 32 experts 99 and 75; 64 experts 180 and 155.  Nine rows:
// 8 experts 30 us single and 44 double, 16 experts 33 and 48, 24 experts 53
// either way).
constexpr int kM4ScheduleThreads = 256;  // the most experts
__global__ __launch_bounds__(kM4ScheduleThreads) void mx4_schedule_kernel(
    const int32_t *__restrict__ offsets, int E, int blocks, int grid, M4Schedule *__restrict__ sch,
    Tile *__restrict__ tiles) {
  constexpr int NC = 5;  // capacities 256, 192, 128, 64, 16
  constexpr int NW = kM4ScheduleThreads / kWave;
  __shared__ int waves[NC][NW];
  const int e = threadIdx.x, lane = lane_id(), wave = threadIdx.x / kWave;
  int row0 = 0, n = 0;
  if (e < E) {
    row0 = offsets[e];
    n = offsets[e + 1] - row0;
  }
  int cap = kTileRows;
  bool many = false;
  for (; cap > 64; cap /= 2) {
    int v = (n + cap - 1) / cap;
#pragma unroll
    for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
    if (lane == 0) waves[0][wave] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) v += waves[0][w];
    __syncthreads();
    many = cap == kTileRows && (long long)v * blocks > grid;
    if ((long long)v * blocks >= grid) break;
  }
  const int full = n / cap, rem = n % cap;
  const int fc = cap == 256 ? 0 : cap == 128 ? 2 : 3;  // class of the full tiles
  const int cls = rem == 0 ? NC : rem > 192 ? 0 : rem > 128 ? 1 : rem > 64 ? 2 : rem > kM4DirectRows ? 3 : 4;
  int at[NC];  // where this expert's tiles of a class begin
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int mine = (c == fc ? full : 0) + (c == cls ? 1 : 0);
    int v = mine;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
      const int x = __shfl_up(v, off);
      if (lane >= off) v += x;
    }
    if (lane == kWave - 1) waves[c][wave] = v;
    at[c] = v - mine;
  }
  __syncthreads();
  int total = 0, last = 0, before = 0;  // all tiles; of the last class; of the one before it
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    at[c] += total;
    before = last;
    last = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < wave) at[c] += waves[c][w];
      last += waves[c][w];
    }
    total += last;
  }
  const int only = n <= cap ? kTileStream : 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    constexpr int kAblk[NC] = {8, 6, 4, 2, 1};
    if (c == fc)
      for (int i = 0; i < full; ++i) tiles[at[c] + i] = Tile{e, row0 + i * cap, cap, kAblk[c] | only};
    if (c == cls)
      tiles[at[c] + (c == fc ? full : 0)] = Tile{e, row0 + full * cap, rem, kAblk[c] | only};
  }
  if (e < 2 * kM4Queues) sch->heads[e / kM4Queues].head[e % kM4Queues] = 0;
  if (e < 2) sch->heads[e].left = 0;
  if (e == 0) {
    sch->n_tiles = total;
    sch->n_small = last;
    sch->n_stream = many ? before : 0;
    sch->many = many;
  }
}

// Work dispatch.  Tile i of the list (tallest first) belongs to queue i % 8,
// and workgroup b to queue b % 8: workgroups go round the eight XCDs in that
// order, so the items of one tile, which share its activation rows, run on
// one XCD and read them through one L2.  A queue is taken from both ends, by
// every other workgroup of an XCD from the back: where a list holds tall
// tiles (bound by the matrix unit) and short ones (weight streams), some
// compute units run the one kind beside the other.
//
// The first item of a workgroup is fixed; more are drawn from the head of
// its queue, which counts draws from the front (low word) and from the back
// (high word), one item ahead so that the draw's latency passes under the
// work.  When its own queue is dry a workgroup looks at all heads at once and
// goes on with a queue that has items left.  The last workgroup to leave
// sets the heads back to zero, as the plan left them: every draw of another
// has returned before that one counts itself out.
struct M4Queues {
  M4Heads *h;
  int nbig, nsmall, ptb, pts;
  int q, G;
  bool back;
  // The state lies in LDS while a workgroup multiplies: the registers are
  // all taken.
  __device__ __forceinline__ M4Queues(M4Heads *h_, const int *state)
      : h(h_), nbig(state[0]), nsmall(state[1]), ptb(state[2]), pts(state[3]), q(state[4]) {
    G = vreg((int)gridDim.x);
    back = (vreg((int)blockIdx.x) / kM4Queues) & 1;
  }
  __device__ __forceinline__ int tall(int p) const { return (nbig - p + kM4Queues - 1) / kM4Queues; }
  __device__ __forceinline__ int items(int p) const {
    const int all = (nbig + nsmall - p + kM4Queues - 1) / kM4Queues, t = tall(p);
    return t * ptb + (all - t) * pts;
  }
  // items of queue p left after v; fixed first items count as drawn
  __device__ __forceinline__ int rest(int p, unsigned long long v) const {
    const int owners = (G - p + kM4Queues - 1) / kM4Queues;
    return items(p) - owners - (int)(uint32_t)v - (int)(v >> 32);
  }
  __device__ __forceinline__ bool item(int i, int *tile, int *part) const {
    const int t = tall(q);
    const int j = i < t * ptb ? i / ptb : t + (i - t * ptb) / pts;
    *part = i < t * ptb ? i - j * ptb : i - t * ptb - (j - t) * pts;
    *tile = q + j * kM4Queues;
    return true;
  }
  __device__ __forceinline__ bool first(int *tile, int *part) const {
    const int rank = vreg((int)blockIdx.x) / kM4Queues / 2, n = items(q);
    if (rank >= (back ? n / 2 : (n + 1) / 2)) return false;
    return item(back ? n - 1 - rank : rank, tile, part);
  }
  // Whether the fixed first items are all there are: nothing is drawn then.
  // Queue 0 has the most items (no fewer tall tiles and no fewer tiles than
  // any other, and a tall tile has no fewer items), queue 7 the fewest owners.
  __device__ __forceinline__ bool fixed() const {
    return items(0) <= G / kM4Queues;
  }
  __device__ __forceinline__ unsigned long long draw() const {
    return atomicAdd(&h->head[q], back ? 1ull << 32 : 1ull);
  }
  // The item that draw() gave, or one of another queue; false if none is left.
  __device__ __forceinline__ bool take(unsigned long long v, int *tile, int *part) {
    for (;;) {
      if (rest(q, v) > 0) {
        const int owners = (G - q + kM4Queues - 1) / kM4Queues;
        const int i = back ? items(q) - 1 - owners / 2 - (int)(v >> 32)
                           : (owners + 1) / 2 + (int)(uint32_t)v;
        return item(i, tile, part);
      }
      unsigned long long heads[kM4Queues];
#pragma unroll
      for (int p = 0; p < kM4Queues; ++p)
        heads[p] = __hip_atomic_load(&h->head[p], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      int most = 0, to = 0;
#pragma unroll
      for (int p = 0; p < kM4Queues; ++p) {
        const int n = rest(p, heads[p]);
        if (n > most) {
          most = n;
          to = p;
        }
      }
      if (most == 0) break;
      q = to;
      v = draw();
    }
    if (atomicAdd(&h->left, 1) == G - 1) {
#pragma unroll
      for (int p = 0; p < kM4Queues; ++p)
        __hip_atomic_store(&h->head[p], 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&h->left, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    return false;
  }
};

template <bool GATEUP>
__global__ __launch_bounds__(kM4Threads, 1) void grouped_gemm_mx4_kernel(Mx4Args a) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kM4Lds];
  // the next item (tile index, first feature; tile -1 = none left) is passed
  // from thread 0 through the idle ring between items
  int *next_item = reinterpret_cast<int *>(ring);
  int *state = reinterpret_cast<int *>(ring + kM4Ring);  // of the dispatch, thread 0's
  const uint32_t ring_lds = lds_addr(ring);
  constexpr int kHalf = GATEUP ? 2 : 1;  // gate and up rows of one feature
  constexpr int FB = kM4WRows / kHalf;  // features per item of the ring
  if (threadIdx.x == 0) {
    const int streamed = m4_stream_takes(a.K) ? a.sch->n_stream : 0;
    // and of tiles of few rows
    const int FS = a.sch->many && (m4_direct_fits(a.K) || streamed) ? 2 * FB : FB;
    state[1] = a.sch->n_small + streamed;
    state[0] = a.sch->n_tiles - state[1];
    state[2] = (a.N + FB - 1) / FB;  // items per tile
    state[3] = (a.N + FS - 1) / FS;
    state[4] = (int)blockIdx.x % kM4Queues;
    state[6] = FS;
    state[7] = a.K;
    state[8] = a.N;
    state[5] = M4Queues(a.heads, state).fixed();
  }
  unsigned long long drawn = 0;
  bool begin = true;
  // the heads from the tile list, at a distance that takes no scalar register
  // (both lie in the workspace, which one int spans between them)
  const int heads_at = vreg((int)(reinterpret_cast<const char *>(a.heads) -
                                  reinterpret_cast<const char *>(a.tiles)));
  const auto heads = [&] {
    return reinterpret_cast<M4Heads *>(reinterpret_cast<char *>(const_cast<Tile *>(a.tiles)) +
                                       heads_at);
  };
  for (;;) {
    if (threadIdx.x == 0) {
      M4Queues queues(heads(), state);
      int ti = -1, part = 0;
      bool some = begin && queues.first(&ti, &part);
      if (!state[5]) {
        if (begin && !some) drawn = queues.draw();
        if (!some) some = queues.take(drawn, &ti, &part);
        state[4] = queues.q;
      }
      begin = false;
      const bool wide = ti >= queues.nbig && state[6] != FB;  // an item of twice the features
      next_item[0] = some ? ti : -1;
      next_item[1] = some ? part * (wide ? 2 * FB : FB) : 0;
      next_item[2] = wide;
    }
    __syncthreads();
    // read before the item's first barrier (its loads overwrite it); the
    // sizes come through LDS so that nothing derived from them is hoisted
    // out of the loop into the scalar registers
    const int ti = __builtin_amdgcn_readfirstlane(next_item[0]);
    if (ti < 0) break;
    const int n0 = __builtin_amdgcn_readfirstlane(next_item[1]);
    Mx4Args ai = a;
    ai.K = __builtin_amdgcn_readfirstlane(state[7]);
    ai.N = __builtin_amdgcn_readfirstlane(state[8]);
    const bool wide = __builtin_amdgcn_readfirstlane(next_item[2]);
    const Tile t = a.tiles[ti];
    if (threadIdx.x == 0 && !state[5])
      drawn = M4Queues(heads(), state).draw();  // for the item after this one
    switch (tile_class(t)) {
      case 8: m4_item<GATEUP, 256>(ai, t, n0, ring, ring_lds); break;
      case 6: m4_item<GATEUP, 192>(ai, t, n0, ring, ring_lds); break;
      case 4: m4_item<GATEUP, 128>(ai, t, n0, ring, ring_lds); break;
      default:
        if (t.nrows <= kM4DirectRows && m4_direct_fits(ai.K)) {
          const int n1 = min(n0 + (wide ? 2 * FB : FB), ai.N);
          if (ai.K % 1024 == 0)
            m4_direct<GATEUP, true>(ai, t, n0, n1, ring);
          else
            m4_direct<GATEUP, false>(ai, t, n0, n1, ring);
        } else if (wide) {
          switch ((t.nrows + 15) / 16) {
            case 4: m4_stream<GATEUP, 4>(ai, t, n0, ring, ring_lds); break;
            case 3: m4_stream<GATEUP, 3>(ai, t, n0, ring, ring_lds); break;
            default: m4_stream<GATEUP, 2>(ai, t, n0, ring, ring_lds); break;
          }
        } else {
          m4_item<GATEUP, 64>(ai, t, n0, ring, ring_lds);
        }
        break;
    }
    // the ring (and the item in it) is rewritten only after every wave has
    // passed this barrier
    __syncthreads();
  }
}

hipError_t launch_ffn_mx4(const FfnLaunchMx4 &L, int stages, hipStream_t stream) {
  M4Schedule *sch = reinterpret_cast<M4Schedule *>(L.sch);
  hipError_t err = hipSuccess;
  if (stages & kStagePlan) {
    err = launch(mx4_schedule_kernel, dim3(1), dim3(kM4ScheduleThreads), stream, L.offsets, L.E,
                 min(L.f / (kM4WRows / 2), (L.d + kM4WRows - 1) / kM4WRows), L.num_cus, sch,
                 L.tiles);
    if (err != hipSuccess) return err;
  }
  Mx4Args g{};
  g.k = L.k;
  g.tiles = L.tiles;
  g.sch = sch;
  if (stages & kStageGateUp) {
    g.act = L.x;
    g.sorted_routes = L.sorted_routes;
    g.w0 = L.wg;
    g.w1 = L.wu;
    g.s0 = L.sg;
    g.s1 = L.su;
    g.out = L.h;
    g.N = L.f;
    g.K = L.d;
    g.heads = &sch->heads[0];
    err = launch(grouped_gemm_mx4_kernel<true>, dim3(L.num_cus), dim3(kM4Threads), stream, g);
    if (err != hipSuccess) return err;
  }
  if (stages & kStageDown) {
    g.act = L.h;
    g.sorted_routes = nullptr;
    g.w0 = L.wd;
    g.w1 = nullptr;
    g.s0 = L.sd;
    g.s1 = nullptr;
    g.out = L.y;
    g.N = L.d;
    g.K = L.f;
    g.heads = &sch->heads[1];
    err = launch(grouped_gemm_mx4_kernel<false>, dim3(L.num_cus), dim3(kM4Threads), stream, g);
  }
  return err;
}

}  // namespace moe

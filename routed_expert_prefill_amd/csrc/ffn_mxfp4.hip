// Persistent grouped GEMM for the routed-MoE FFN with MXFP4 weights (mx4.h)
// and bf16 activations: one kernel per projection (gate/up with the SwiGLU
// epilogue, then down), fp32 accumulation.
//
// Same tile list, two work queues and direct global->LDS stage ring as the
// bf16 kernels (ffn_grouped.hip, ring.h).  The ring holds the weights as
// codes, a quarter of the bf16 bytes; a wave reads 16 bytes of a weight row
// per lane -- 32 codes, exactly one scale group -- and converts them in
// registers in front of the MFMAs, so no pass over expanded weights exists.
// The order of the reduction inside a stage follows from that: lane half h
// of a 64-column step holds group h of it, and MFMA j of the step multiplies
// columns 8 j .. 8 j + 7 of both groups.
//
// A stage is KB blocks of 64 columns: the activation rows' 128-byte lines of
// each block, 32 KB bytes of codes per weight row, and the groups' scales.
// KB = 4 makes the codes of a row whole 128-byte lines, which HBM streams at
// full rate; tall tiles, bound by the matrix unit and re-reading weights
// through the caches, take KB = 1 so that three stages fit in LDS.
#include "kernels.h"
#include "mx4.h"
#include "ring.h"

namespace moe {

struct Mx4Args {
  const uint16_t *act;           // gate/up: x [T, K]; down: h [R, K]
  const int32_t *sorted_routes;  // gate/up: token of sorted row i is sorted_routes[i] / k
  int k;
  const uint8_t *w0, *w1;  // codes [E, N, K / 2]: gate (or down), up
  const uint8_t *s0, *s1;  // scales [E, N, K / 32] of w0, w1
  void *out;               // gate/up: h bf16 [R, N]; down: y fp32 [R, N]
  int N, K;
  const Tile *tiles;
  const int *ntiles;
  const int *n_small;  // 32-row tiles at the end of the tile list
  const int *n_multi;  // tiles of experts with several tiles, at the start of the list
  int *counter;        // compute-queue head (TwoQueue), zeroed by the schedule
  int *counter_s;      // stream-queue head
};

constexpr int kM4Threads = 512;
constexpr int kM4Waves = kM4Threads / kWave;
constexpr int kM4Ring = 160 * 1024;  // the whole LDS of a workgroup

// Geometry of an item with AR activation rows, WR weight rows and KB
// 64-column blocks per stage.
template <int AR, int WR, int KB>
struct M4Ring {
  static constexpr int kAct = AR * 128 * KB;
  static constexpr int kCodes = WR * 32 * KB;
  static constexpr int kScaleRow = KB == 4 ? 8 : 4;  // bytes of scales per weight row
  static constexpr int kSlot = kAct + kCodes + WR * kScaleRow;
  // tiles of at most 32 rows: waves 4-7 hand their sums to waves 0-3 behind the ring
  static constexpr int kSums = AR <= 32 ? 4 * 4096 : 0;
  static constexpr int kFit = (kM4Ring - kSums) / kSlot;
  static constexpr int kDepth = kFit < 8 ? kFit : 8;
};

// 16-byte chunk c of the codes of weight row r is stored at this slot of the
// row's 2 KB: 16 lanes reading one chunk of 16 consecutive rows then touch
// 16 distinct 16-byte slots of a 256-byte window.
template <int KB>
__device__ __forceinline__ int m4_slot(int r, int c) {
  return c ^ ((r / (8 / KB)) & (2 * KB - 1));
}

// Direct global->LDS load of 4 bytes per lane to LDS byte address
// lds_byte_addr + 4 * lane (see dma16).
__device__ __forceinline__ void dma4(const void *src, uint32_t lds_byte_addr) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(lds_byte_addr)
               : "memory");
}

// Wave wv multiplies TT activation tiles by TW weight tiles of 32 rows.  With
// at most 32 activation rows (and 128 weight rows) four waves would do, so
// the other four take the second half of each stage's columns.
template <int AR>
struct M4Layout {
  static constexpr bool kSplit = AR <= 32;
  static constexpr int TT = kSplit ? 1 : AR / 64;
  static constexpr int TW = kSplit ? 1 : 2;
  __device__ static int atile(int wv, int tt) { return kSplit ? 0 : (wv >> 2) * TT + tt; }
  __device__ static int wtile(int wv, int tw) { return kSplit ? (wv & 3) : (wv & 3) * 2 + tw; }
};

__device__ __forceinline__ f32x4 m4_quad(const f32x16 &v, int g) {
  return f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
}

// nb feature blocks of one tile, streamed through one ring fill.
// NT: codes through non-temporal loads (whole lines only: KB == 4).
template <bool GATEUP, bool NT, int AR, int WR, int KB>
__device__ __forceinline__ void m4_item(const Mx4Args &a, const Tile &t, int n0, int nb_arg,
                                        uint8_t *ring, uint32_t ring_lds) {
  static_assert(!NT || KB == 4, "half lines must not bypass the caches");
  using L = M4Layout<AR>;
  using G = M4Ring<AR, WR, KB>;
  static_assert(L::kSplit ? WR == 128 && KB == 4 : WR == 256 && AR % 64 == 0, "wave layout");
  constexpr bool MB = L::kSplit;  // several blocks only where items are short
  constexpr int FEAT = GATEUP ? WR / 2 : WR;  // output features per block
  constexpr int TT = L::TT, TW = L::TW;
  constexpr int NA = KB * AR / 8;      // activation loads: 8 rows of 128 bytes
  constexpr int NW = WR * KB / 32;     // code loads: 1 KB
  constexpr int NC = G::kScaleRow * WR / 256;  // scale loads: 256 bytes
  // load i of a kind goes to wave i % 8, the loads of scales to the last NC waves
  static_assert((NA % kM4Waves == 0 || NA < kM4Waves) && NW % kM4Waves == 0 && NC <= kM4Waves,
                "shares");
  constexpr int JA = (NA + kM4Waves - 1) / kM4Waves, JW = NW / kM4Waves;
  constexpr int NS = G::kDepth;
  static_assert(NS >= 2 && (JA + JW + 1) * (NS - 2) <= 32, "wait_vm counts to 32");
  const int nb = MB ? nb_arg : 1;
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int K = a.K;
  const int nst = (K / 64 + KB - 1) / KB;
  const bool half = KB == 4 && (K & 128) != 0;  // the last stage has two blocks only
  const bool has_act = NA % kM4Waves == 0 || wv < NA, has_scales = wv >= kM4Waves - NC;
  const int cnt = JW + (has_act ? JA : 0) + (has_scales ? 1 : 0);  // loads of this wave per stage

  auto wrow = [&](int wr, const uint8_t *p0, const uint8_t *p1, int row_bytes) {
    const uint8_t *w = p0;
    int n;
    if (GATEUP) {  // 16-row groups alternate gate and up
      if ((wr >> 4) & 1) w = p1;
      n = n0 + (wr >> 5) * 16 + (wr & 15);
    } else {
      n = min(n0 + wr, a.N - 1);
    }
    return w + ((size_t)t.e * a.N + n) * row_bytes;
  };
  // this lane's source of each of its loads at stage 0.  In a half stage the
  // sources of the missing second half move back to the first (loaded, not used).
  const uint8_t *act[JA], *codes[JW], *scales;
#pragma unroll
  for (int j = 0; j < JA; ++j) {
    const int i = wv + kM4Waves * j;
    const int kb = i / (AR / 8);
    const int r = (i - kb * (AR / 8)) * 8 + (lane >> 3);
    const int row = t.row0 + min(r, t.nrows - 1);
    const size_t s = GATEUP ? (size_t)(a.sorted_routes[row] / a.k) : (size_t)row;
    act[j] = reinterpret_cast<const uint8_t *>(a.act + s * K) + kb * 128 +
             ring_slot(r, lane & 7) * 16;
  }
  constexpr int LPR = 2 * KB;  // lanes per row of codes
  int code_back = 0;
#pragma unroll
  for (int j = 0; j < JW; ++j) {
    const int r = (wv + kM4Waves * j) * (64 / LPR) + lane / LPR;
    const int c = m4_slot<KB>(r, lane % LPR);
    codes[j] = wrow(r, a.w0, a.w1, K / 2) + c * 16;
    code_back |= (c >= 4 ? 1 : 0) << j;
  }
  {
    constexpr int SPR = G::kScaleRow / 4;  // lanes per row of scales
    const int i = max(wv - (kM4Waves - NC), 0);
    scales = wrow(i * (64 / SPR) + lane / SPR, a.s0, a.s1, K / 32) + (lane % SPR) * 4;
  }
  // loads of stage s of block b
  auto issue = [&](int s, int b, int slot) {
    const uint32_t base = ring_lds + (uint32_t)(slot * G::kSlot) + (uint32_t)wv * 1024u;
    const bool cut = half && s == nst - 1;
    const uint32_t act_off = (uint32_t)s * (128 * KB);
    const uint32_t code_off = (uint32_t)s * (32 * KB) + (MB ? (uint32_t)(b * FEAT) * (K / 2) : 0);
    if (has_act) {
#pragma unroll
      for (int j = 0; j < JA; ++j) {
        const uint8_t *p = act[j] + act_off;
        if (KB == 4 && cut && (wv + kM4Waves * j) / (AR / 8) >= 2) p -= 256;
        dma16(p, base + (uint32_t)j * (kM4Waves * 1024u));
      }
    }
#pragma unroll
    for (int j = 0; j < JW; ++j) {
      const uint8_t *p = codes[j] + code_off;
      if (KB == 4 && cut) p -= ((code_back >> j) & 1) * 64;
      const uint32_t to = base + (uint32_t)G::kAct + (uint32_t)j * (kM4Waves * 1024u);
      if (NT)
        dma16_nt(p, to);
      else
        dma16(p, to);
    }
    if (has_scales) {
      // two scales per block; KB == 1 loads the aligned four that hold them
      const uint8_t *p = scales + (KB == 1 ? (s >> 1) * 4 : s * (2 * KB)) +
                         (MB ? (uint32_t)(b * FEAT) * (K / 32) : 0);
      if (KB == 4 && cut) p -= (lane & 1) * 4;
      dma4(p, ring_lds + (uint32_t)(slot * G::kSlot + G::kAct + G::kCodes) +
                  (uint32_t)(wv - (kM4Waves - NC)) * 256u);
    }
  };

  const int rr = lane & 31, rh = lane >> 5;
  f32x16 acc[TW][TT];
  auto zero_acc = [&]() {
#pragma unroll
    for (int tw = 0; tw < TW; ++tw)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[tw][tt][j] = 0.f;
  };

  // the MFMAs of one ring stage
  auto mma_stage = [&](const uint8_t *buf, int s) {
    static_assert(L::kSplit || KB <= 2, "one word of scales per wave and stage");
    uint32_t sc[TW];
#pragma unroll
    for (int tw = 0; tw < TW; ++tw) {
      const uint8_t *p = buf + G::kAct + G::kCodes + (L::wtile(wv, tw) * 32 + rr) * G::kScaleRow;
      if (L::kSplit) p += (wv >> 2) * 4;
      sc[tw] = *reinterpret_cast<const uint32_t *>(p) >> (8 * rh + (KB == 1 ? 16 * (s & 1) : 0));
    }
    if (L::kSplit && wv >= 4 && half && s == nst - 1) return;  // no second half there
    constexpr int KW = L::kSplit ? KB / 2 : KB;  // blocks of this wave
#pragma unroll
    for (int q = 0; q < KW; ++q) {
      const int kb = L::kSplit ? (wv >> 2) * 2 + q : q;
      i32x4 raw[TW];
      float scale[TW];
#pragma unroll
      for (int tw = 0; tw < TW; ++tw) {
        const int r = L::wtile(wv, tw) * 32 + rr;
        raw[tw] = *reinterpret_cast<const i32x4 *>(buf + G::kAct + r * (32 * KB) +
                                                   m4_slot<KB>(r, 2 * kb + rh) * 16);
        scale[tw] = mx4_scale((sc[tw] >> (16 * (q & 1))) & 0xffu);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 fa[TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const int r = (L::atile(wv, tt) * 32 + rr) & (AR < 32 ? AR - 1 : -1);
          fa[tt] = *reinterpret_cast<const bf16x8 *>(buf + kb * (AR * 128) + r * 128 +
                                                     ring_slot(r, 4 * rh + j) * 16);
        }
#pragma unroll
        for (int tw = 0; tw < TW; ++tw) {
          const bf16x8 fw = mx4_decode8((uint32_t)raw[tw][j], scale[tw]);
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) acc[tw][tt] = mfma32_bf16(fw, fa[tt], acc[tw][tt]);
        }
      }
    }
  };

  // results of the block at feature nb0
  auto epilogue = [&](int nb0) {
    if constexpr (L::kSplit) {
      f32x4 *sums = reinterpret_cast<f32x4 *>(ring + kM4Ring - G::kSums) + (wv & 3) * 256 + lane;
      if (wv >= 4) {
#pragma unroll
        for (int g = 0; g < 4; ++g) sums[g * 64] = m4_quad(acc[0][0], g);
      }
      // the sums are written; the next ones are a barrier of every stage away
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      ring_barrier();
      if (wv >= 4) return;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 v = sums[g * 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[0][0][4 * g + i] += v[i];
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
            const int n = nb0 + wt * 16 + g * 8 + rh * 4;
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
            const int n = nb0 + wt * 32 + g * 8 + rh * 4;
            if (n < a.N)
              *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + row * a.N + n) =
                  m4_quad(acc[tw][tt], g);
          }
        }
      }
    }
  };

  zero_acc();
  wait_vm(0);
  ring_barrier();  // every wave is done with the ring contents of the previous item
  const int total = MB ? nb * nst : nst;
  int is = 0, ib = 0;  // stage and block of the next stage to load
  auto issue_next = [&](int slot) {
    issue(is, ib, slot);
    if (++is == nst && MB) {
      is = 0;
      ++ib;
    }
  };
#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < total) issue_next(s);
  int slot = 0, cs = 0, cb = 0;  // stage and block being multiplied
  for (int s = 0; s < total; ++s) {
    // this wave's loads of stage s are done; later stages may stay in flight
    // (stores of an earlier block, counted too, only make the wait longer)
    wait_vm(cnt * min(NS - 2, total - 1 - s));
    ring_barrier();  // stage s is in LDS for everyone; stage s - 1 is consumed
    if (s + NS - 1 < total) issue_next(slot == 0 ? NS - 1 : slot - 1);
    mma_stage(ring + slot * G::kSlot, MB ? cs : s);
    slot = slot == NS - 1 ? 0 : slot + 1;
    if (MB && ++cs == nst) {
      epilogue(n0 + cb * FEAT);
      cs = 0;
      if (++cb < nb) zero_acc();
    }
  }
  if (!MB) epilogue(n0);
}

// A pointer through two words of LDS.
__device__ __forceinline__ void m4_put(int *to, const void *p) {
  const uint64_t v = (uint64_t)(uintptr_t)p;
  to[0] = (int)(uint32_t)v;
  to[1] = (int)(uint32_t)(v >> 32);
}
__device__ __forceinline__ void *m4_get(const int *from) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane(from[0]);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane(from[1]);
  return reinterpret_cast<void *>((uintptr_t)(((uint64_t)hi << 32) | lo));
}

// Weight rows per item: 256, and 128 for 32-row tiles.
constexpr int kM4WRows = 256;
constexpr int kM4WRowsSmall = 128;

template <bool GATEUP>
__global__ __launch_bounds__(kM4Threads, 1) void grouped_gemm_mx4_kernel(Mx4Args a) {
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kM4Ring];
  // the next item (tile index, first feature; tile -1 = none left) is passed
  // from thread 0 through the idle ring between items
  int *next_item = reinterpret_cast<int *>(ring);
  const uint32_t ring_lds = lds_addr(ring);
  constexpr int kHalf = GATEUP ? 2 : 1;  // gate and up rows of one feature
  constexpr int FB = kM4WRows / kHalf, FS = kM4WRowsSmall / kHalf;  // features per item
  const int N = vreg(a.N);
  const int grid = vreg((int)gridDim.x);
  const int nsmall = vreg(*a.n_small), nbig = vreg(*a.ntiles) - nsmall;
  const int ptb = (N + FB - 1) / FB, pts = N / FS;  // blocks of a tile
  // 32-row tiles: four (two) blocks per item while every workgroup gets two
  // items, and single ones at the end of the list, about two rounds of them
  int nbs = pts % 4 == 0 ? 4 : pts % 2 == 0 ? 2 : 1;
  while (nbs > 1 && nsmall * (pts / nbs) < 2 * grid) nbs >>= 1;
  const int ntail = nbs > 1 ? min(nsmall, (2 * grid + pts - 1) / pts) : 0;
  const int ptm = pts / nbs;
  const int items_big = nbig * ptb, items_mid = items_big + (nsmall - ntail) * ptm;
  const int total = items_mid + ntail * pts;
  TwoQueue queue(vreg(*a.n_multi) * ptb, total, GATEUP ? 6 : 9, grid);
  for (;;) {
    if (threadIdx.x == 0) {
      const int it = queue.next(a.counter, a.counter_s);
      int ti = -1, n0 = 0, nb = 1;
      if (it < items_big) {
        ti = it / ptb;
        n0 = (it - ti * ptb) * FB;
      } else if (it < items_mid) {
        const int q = (it - items_big) / ptm;
        ti = nbig + q;
        n0 = (it - items_big - q * ptm) * FS * nbs;
        nb = nbs;
      } else if (it < total) {
        const int q = (it - items_mid) / pts;
        ti = nbig + nsmall - ntail + q;
        n0 = (it - items_mid - q * pts) * FS;
      }
      next_item[3] = nb;
      next_item[0] = ti;
      next_item[1] = n0;
      next_item[2] = a.K;
      m4_put(next_item + 4, a.s0);
      m4_put(next_item + 6, a.s1);
      m4_put(next_item + 8, a.out);
    }
    __syncthreads();
    // read before the item's first barrier (its loads overwrite it); the
    // reduction length and some of the pointers come through LDS so that
    // they, and what derives from them, are not held in scalar registers
    // across the loop (they do not fit)
    const int ti = __builtin_amdgcn_readfirstlane(next_item[0]);
    if (ti < 0) break;
    const int n0 = __builtin_amdgcn_readfirstlane(next_item[1]);
    Mx4Args ai = a;
    ai.K = __builtin_amdgcn_readfirstlane(next_item[2]);
    ai.s0 = static_cast<const uint8_t *>(m4_get(next_item + 4));
    ai.s1 = static_cast<const uint8_t *>(m4_get(next_item + 6));
    ai.out = m4_get(next_item + 8);
    const Tile t = a.tiles[ti];
    const int nb = __builtin_amdgcn_readfirstlane(next_item[3]);
    switch (tile_class(t)) {
      case 8: m4_item<GATEUP, false, 256, kM4WRows, 1>(ai, t, n0, 1, ring, ring_lds); break;
      case 6: m4_item<GATEUP, false, 192, kM4WRows, 1>(ai, t, n0, 1, ring, ring_lds); break;
      case 4: m4_item<GATEUP, false, 128, kM4WRows, 2>(ai, t, n0, 1, ring, ring_lds); break;
      case 2: m4_item<GATEUP, false, 64, kM4WRows, 2>(ai, t, n0, 1, ring, ring_lds); break;
      default:
        if (!(t.ablk & kTileStream))
          m4_item<GATEUP, false, 32, kM4WRowsSmall, 4>(ai, t, n0, nb, ring, ring_lds);
        else if (t.nrows > 16)
          m4_item<GATEUP, true, 32, kM4WRowsSmall, 4>(ai, t, n0, nb, ring, ring_lds);
        else if (t.nrows > 8)
          m4_item<GATEUP, true, 16, kM4WRowsSmall, 4>(ai, t, n0, nb, ring, ring_lds);
        else
          m4_item<GATEUP, true, 8, kM4WRowsSmall, 4>(ai, t, n0, nb, ring, ring_lds);
        break;
    }
    // the ring (and the item in it) is rewritten only after every wave has
    // passed this barrier
    __syncthreads();
  }
}

hipError_t launch_ffn_mx4(const FfnLaunchMx4 &L, int stages, hipStream_t stream) {
  if (stages & kStagePlan) {
    const hipError_t err = launch_grouped_schedule(L.offsets, L.E, L.sch, L.tiles, stream);
    if (err != hipSuccess) return err;
  }
  Mx4Args g{};
  g.k = L.k;
  g.tiles = L.tiles;
  g.ntiles = &L.sch->n_tiles;
  g.n_small = &L.sch->n_small;
  g.n_multi = &L.sch->n_multi;
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
    g.counter = &L.sch->counter[0];
    g.counter_s = &L.sch->counter_s[0];
    hipLaunchKernelGGL(grouped_gemm_mx4_kernel<true>, dim3(L.num_cus), dim3(kM4Threads), 0, stream,
                       g);
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
    g.counter = &L.sch->counter[1];
    g.counter_s = &L.sch->counter_s[1];
    hipLaunchKernelGGL(grouped_gemm_mx4_kernel<false>, dim3(L.num_cus), dim3(kM4Threads), 0,
                       stream, g);
  }
  return hipGetLastError();
}

}  // namespace moe

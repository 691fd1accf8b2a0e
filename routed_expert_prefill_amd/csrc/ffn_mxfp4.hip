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

// Geometry of an item with 32 * AB activation rows, WR weight rows and KB
// 64-column blocks per stage.
template <int AB, int WR, int KB>
struct M4Ring {
  static constexpr int kAct = 32 * AB * 128 * KB;
  static constexpr int kCodes = WR * 32 * KB;
  static constexpr int kScaleRow = KB == 4 ? 8 : 4;  // bytes of scales per weight row
  static constexpr int kSlot = kAct + kCodes + WR * kScaleRow;
  static constexpr int kDepth = (kM4Ring / kSlot) < 8 ? (kM4Ring / kSlot) : 8;
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

// Wave wv multiplies TT activation tiles by TW weight tiles of 32 rows.
template <int AB, int WR>
struct M4Layout {
  static constexpr int TT = AB == 1 ? 1 : AB / 2;
  static constexpr int TW = AB == 1 ? 1 : 2;
  __device__ static bool active(int wv) { return AB > 1 || wv < WR / 32; }
  __device__ static int atile(int wv, int tt) { return AB == 1 ? 0 : (wv >> 2) * TT + tt; }
  __device__ static int wtile(int wv, int tw) { return AB == 1 ? wv : (wv & 3) * 2 + tw; }
};

__device__ __forceinline__ f32x4 m4_quad(const f32x16 &v, int g) {
  return f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
}

// NT: codes through non-temporal loads (whole lines only: KB == 4).
template <bool GATEUP, bool NT, int AB, int WR, int KB>
__device__ __forceinline__ void m4_item(const Mx4Args &a, const Tile &t, int n0, uint8_t *ring,
                                        uint32_t ring_lds) {
  static_assert(!NT || KB == 4, "half lines must not bypass the caches");
  static_assert(AB == 1 || WR == 256, "taller tiles take 256 weight rows");
  using L = M4Layout<AB, WR>;
  using G = M4Ring<AB, WR, KB>;
  constexpr int TT = L::TT, TW = L::TW;
  constexpr int NA = KB * 4 * AB;      // activation loads: 8 rows of 128 bytes
  constexpr int NW = WR * KB / 32;     // code loads: 1 KB
  constexpr int NC = G::kScaleRow * WR / 256;  // scale loads: 256 bytes
  // load i of a kind goes to wave i % 8: JA + JW loads of every wave and one
  // load of scales of the first NC waves per stage
  static_assert(NA % kM4Waves == 0 && NW % kM4Waves == 0 && NC <= kM4Waves, "even shares");
  constexpr int JA = NA / kM4Waves, JW = NW / kM4Waves;
  constexpr int NS = G::kDepth;
  static_assert(NS >= 2 && (JA + JW + 1) * (NS - 2) <= 32, "wait_vm counts to 32");
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int K = a.K;
  const int nst = (K / 64 + KB - 1) / KB;
  const bool half = KB == 4 && (K & 128) != 0;  // the last stage has two blocks only
  const int cnt = JA + JW + (wv < NC ? 1 : 0);  // loads this wave issues per stage

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
    const int kb = i / (4 * AB);
    const int r = (i - kb * 4 * AB) * 8 + (lane >> 3);
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
    scales = wrow(min(wv, NC - 1) * (64 / SPR) + lane / SPR, a.s0, a.s1, K / 32) + (lane % SPR) * 4;
  }
  auto issue = [&](int s, int slot) {
    const uint32_t base = ring_lds + (uint32_t)(slot * G::kSlot) + (uint32_t)wv * 1024u;
    const bool cut = half && s == nst - 1;
    const uint32_t act_off = (uint32_t)s * (128 * KB), code_off = (uint32_t)s * (32 * KB);
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      const uint8_t *p = act[j] + act_off;
      if (KB == 4 && cut && (wv + kM4Waves * j) / (4 * AB) >= 2) p -= 256;
      dma16(p, base + (uint32_t)j * (kM4Waves * 1024u));
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
    if (wv < NC) {
      // two scales per block; KB == 1 loads the aligned four that hold them
      const uint8_t *p = scales + (KB == 1 ? (s >> 1) * 4 : s * (2 * KB));
      if (KB == 4 && cut) p -= (lane & 1) * 4;
      dma4(p, ring_lds + (uint32_t)(slot * G::kSlot + G::kAct + G::kCodes) + (uint32_t)wv * 256u);
    }
  };

  const int rr = lane & 31, rh = lane >> 5;
  f32x16 acc[TW][TT];
#pragma unroll
  for (int tw = 0; tw < TW; ++tw)
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[tw][tt][j] = 0.f;

  auto mma_stage = [&](const uint8_t *buf, int s) {
    if (!L::active(wv)) return;
    uint32_t sc[TW][KB == 4 ? 2 : 1];
#pragma unroll
    for (int tw = 0; tw < TW; ++tw) {
      const uint8_t *p = buf + G::kAct + G::kCodes + (L::wtile(wv, tw) * 32 + rr) * G::kScaleRow;
      if constexpr (KB == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        sc[tw][0] = v.x >> (8 * rh);
        sc[tw][1] = v.y >> (8 * rh);
      } else {
        sc[tw][0] = *reinterpret_cast<const uint32_t *>(p) >> (8 * rh + (KB == 1 ? 16 * (s & 1) : 0));
      }
    }
    const int blocks = half && s == nst - 1 ? 2 : KB;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kb >= blocks) break;
      i32x4 raw[TW];
      float scale[TW];
#pragma unroll
      for (int tw = 0; tw < TW; ++tw) {
        const int r = L::wtile(wv, tw) * 32 + rr;
        raw[tw] = *reinterpret_cast<const i32x4 *>(buf + G::kAct + r * (32 * KB) +
                                                   m4_slot<KB>(r, 2 * kb + rh) * 16);
        scale[tw] = mx4_scale((sc[tw][kb >> 1] >> (16 * (kb & 1))) & 0xffu);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 fa[TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const int r = L::atile(wv, tt) * 32 + rr;
          fa[tt] = *reinterpret_cast<const bf16x8 *>(buf + kb * (32 * AB * 128) + r * 128 +
                                                     ring_slot(rr, 4 * rh + j) * 16);
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

  wait_vm(0);
  ring_barrier();  // every wave is done with the ring contents of the previous item
#pragma unroll
  for (int s = 0; s < NS - 1; ++s)
    if (s < nst) issue(s, s);
  int slot = 0;
  for (int s = 0; s < nst; ++s) {
    // this wave's loads of stage s are done; later stages may stay in flight
    wait_vm(cnt * min(NS - 2, nst - 1 - s));
    ring_barrier();  // stage s is in LDS for everyone; stage s - 1 is consumed
    const int ahead = s + NS - 1;
    if (ahead < nst) issue(ahead, slot == 0 ? NS - 1 : slot - 1);
    mma_stage(ring + slot * G::kSlot, s);
    slot = slot == NS - 1 ? 0 : slot + 1;
  }
  if (!L::active(wv)) return;
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
  const int nsmall = vreg(*a.n_small), nbig = vreg(*a.ntiles) - nsmall;
  const int ptb = (N + FB - 1) / FB, pts = (N + FS - 1) / FS;
  const int items_big = nbig * ptb, total = items_big + nsmall * pts;
  TwoQueue queue(vreg(*a.n_multi) * ptb, total, GATEUP ? 6 : 9, vreg((int)gridDim.x));
  for (;;) {
    if (threadIdx.x == 0) {
      const int it = queue.next(a.counter, a.counter_s);
      int ti = -1, n0 = 0;
      if (it < items_big) {
        ti = it / ptb;
        n0 = (it - ti * ptb) * FB;
      } else if (it < total) {
        const int q = (it - items_big) / pts;
        ti = nbig + q;
        n0 = (it - items_big - q * pts) * FS;
      }
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
    switch (tile_class(t)) {
      case 8: m4_item<GATEUP, false, 8, kM4WRows, 1>(ai, t, n0, ring, ring_lds); break;
      case 6: m4_item<GATEUP, false, 6, kM4WRows, 1>(ai, t, n0, ring, ring_lds); break;
      case 4: m4_item<GATEUP, false, 4, kM4WRows, 2>(ai, t, n0, ring, ring_lds); break;
      case 2: m4_item<GATEUP, false, 2, kM4WRows, 2>(ai, t, n0, ring, ring_lds); break;
      default:
        if (t.ablk & kTileStream)
          m4_item<GATEUP, true, 1, kM4WRowsSmall, 4>(ai, t, n0, ring, ring_lds);
        else
          m4_item<GATEUP, false, 1, kM4WRowsSmall, 4>(ai, t, n0, ring, ring_lds);
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

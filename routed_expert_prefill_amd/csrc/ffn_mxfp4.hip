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

constexpr int kM4Queues = 8;

// Heads of a projection's work queues, and the workgroups that have left.
struct M4Heads {
  unsigned long long head[kM4Queues];
  int left, pad;
};

// What the plan leaves at the start of the workspace.
struct M4Schedule {
  int n_tiles;  // entries of the tile list, tallest capacity first
  int n_small;  // 32-row tiles, the last n_small entries
  int pad[2];
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
  const int *ntiles;
  const int *n_small;  // 32-row tiles at the end of the tile list
  M4Heads *heads;      // of the work queues (M4Queues), zeroed by the plan
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
  static constexpr int kSlot = kAct + kCodes;
  // Scales come in groups of 16 bytes per weight row, for kGroup stages.  A
  // group is loaded with its first stage and read until its last, so two
  // buffers do if a group is at least as long as the ring (less one stage);
  // items of several blocks, whose groups end with each block, have one
  // buffer per slot.
  static constexpr int kGroup = 8 / KB;
  static constexpr int kScales = WR * 16;
  static constexpr bool kSmall = AR <= 32;
  // small tiles: waves 4-7 hand their sums to waves 0-3 behind the ring
  static constexpr int kSums = kSmall ? 4 * 4096 : 0;
  static constexpr int kFit = kSmall ? (kM4Ring - kSums) / (kSlot + kScales)
                                     : (kM4Ring - 2 * kScales) / kSlot;
  static constexpr int kDepth = kFit < 8 ? kFit : 8;
  static constexpr int kBuffers = kSmall ? kDepth : 2;
  static_assert(kSmall || kGroup >= kDepth - 1, "two buffers of scales");
  static constexpr int kScaleBase = kDepth * kSlot;
  static_assert(kScaleBase + kBuffers * kScales + kSums <= kM4Ring, "fits");
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
  // load i of a kind goes to wave i % 8
  static_assert(NA % kM4Waves == 0 && NW % kM4Waves == 0, "even shares");
  constexpr int JA = NA / kM4Waves, JW = NW / kM4Waves;
  constexpr int NS = G::kDepth;
  static_assert(NS >= 2 && (JA + JW) * (NS - 2) <= 32, "wait_vm counts to 32");
  const int nb = MB ? nb_arg : 1;
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int K = a.K;
  const int nst = (K / 64 + KB - 1) / KB;
  const bool half = KB == 4 && (K & 128) != 0;  // the last stage has two blocks only
  // loads of this wave per stage, scales left out: where they are in flight
  // the wait below ends a load later than it has to
  const int cnt = JA + JW;

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
  const uint8_t *act[JA], *codes[JW];
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
  // Scales of a group: where rows start on 16-byte borders, one load of 16
  // bytes per lane and 64 rows by each of the last WR / 64 waves; elsewhere
  // loads of 4 bytes per lane and 16 rows.  Both leave 16 bytes per row in LDS.
  constexpr int SW = WR / 64;
  const bool wide = (K & 511) == 0;
  const int swv = wv - (kM4Waves - SW);
  const int srow = wide ? max(swv, 0) * 64 + lane : wv * (WR / 8) + (lane >> 2);
  const uint8_t *scales = wrow(srow, a.s0, a.s1, K / 32);
  int group = 0;  // groups loaded so far
  auto issue_scales = [&](int s, int b) {
    const uint32_t to = ring_lds + (uint32_t)G::kScaleBase +
                        (unsigned)group % (unsigned)G::kBuffers * G::kScales;
    ++group;
    uint32_t off = (uint32_t)s * (2 * KB) + (MB ? (uint32_t)(b * FEAT) * (K / 32) : 0);
    if (wide) {
      if (swv >= 0) dma16(scales + off, to + (uint32_t)swv * 1024u);
    } else {
      // words past the row's end are not there: the group's first instead
      off += (s * KB + (lane & 3) * 2) * 64 < K ? (lane & 3) * 4 : 0;
      dma4(scales + off, to + (uint32_t)wv * (WR * 2u));
      if (WR == 256)
        dma4(wrow(srow + 16, a.s0, a.s1, K / 32) + off, to + (uint32_t)wv * (WR * 2u) + 256u);
    }
  };
  // loads of stage s of block b
  auto issue = [&](int s, int b, int slot) {
    const uint32_t base = ring_lds + (uint32_t)(slot * G::kSlot) + (uint32_t)wv * 1024u;
    const bool cut = half && s == nst - 1;
    const uint32_t act_off = (uint32_t)s * (128 * KB);
    const uint32_t code_off = (uint32_t)s * (32 * KB) + (MB ? (uint32_t)(b * FEAT) * (K / 2) : 0);
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      const uint8_t *p = act[j] + act_off;
      if (KB == 4 && cut && (wv + kM4Waves * j) / (AR / 8) >= 2) p -= 256;
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
    if (s % G::kGroup == 0) issue_scales(s, b);
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

  // the MFMAs of one ring stage; sbuf: the buffer with its group of scales
  auto mma_stage = [&](const uint8_t *buf, const uint8_t *sbuf, int s) {
    if (L::kSplit && wv >= 4 && half && s == nst - 1) return;  // no second half there
    constexpr int KW = L::kSplit ? KB / 2 : KB;  // blocks of this wave
    const int kb0 = L::kSplit ? (wv >> 2) * 2 : 0;
    // two scales per block and four to a word: the word of this wave's blocks
    const int word = L::kSplit ? (s & 1) * 2 + (wv >> 2) : KB == 2 ? s & 3 : (s >> 1) & 3;
    uint32_t sc[TW];
    i32x4 raw[KW][TW];
#pragma unroll
    for (int tw = 0; tw < TW; ++tw) {
      const int r = L::wtile(wv, tw) * 32 + rr;
      sc[tw] = *reinterpret_cast<const uint32_t *>(sbuf + r * 16 + word * 4) >>
               (8 * rh + (KB == 1 ? 16 * (s & 1) : 0));
#pragma unroll
      for (int q = 0; q < KW; ++q)
        raw[q][tw] = *reinterpret_cast<const i32x4 *>(
            buf + G::kAct + r * (32 * KB) + m4_slot<KB>(r, 2 * (kb0 + q) + rh) * 16);
    }
    auto load_act = [&](int q, int j, bf16x8 (&fa)[TT]) {
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const int r = L::atile(wv, tt) * 32 + rr;
        fa[tt] = *reinterpret_cast<const bf16x8 *>(buf + (kb0 + q) * (AR * 128) + r * 128 +
                                                   ring_slot(r, 4 * rh + j) * 16);
      }
    };
    if constexpr (L::kSplit) {
      // everything the stage needs is read ahead: with one tile pair per wave
      // a read in front of each MFMA left the wave waiting for LDS most of
      // the time
      bf16x8 fa[KW][4][TT];
#pragma unroll
      for (int q = 0; q < KW; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) load_act(q, j, fa[q][j]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < KW; ++q) {
        const float scale = mx4_scale((sc[0] >> (16 * q)) & 0xffu);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[0][0] = mfma32_bf16(mx4_decode8((uint32_t)raw[q][0][j], scale), fa[q][j][0], acc[0][0]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < KW; ++q) {
        float scale[TW];
#pragma unroll
        for (int tw = 0; tw < TW; ++tw) scale[tw] = mx4_scale((sc[tw] >> (16 * q)) & 0xffu);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x8 fa[TT];
          load_act(q, j, fa);
#pragma unroll
          for (int tw = 0; tw < TW; ++tw) {
            const bf16x8 fw = mx4_decode8((uint32_t)raw[q][tw][j], scale[tw]);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) acc[tw][tt] = mfma32_bf16(fw, fa[tt], acc[tw][tt]);
          }
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
  ring_barrier();  // every wave has read its item, which lies in the ring
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
  int cg = 0;                    // buffer of its group of scales
  for (int s = 0; s < total; ++s) {
    // this wave's loads of stage s are done; later stages may stay in flight
    // (stores of an earlier block, counted too, only make the wait longer)
    wait_vm(cnt * min(NS - 2, total - 1 - s));
    ring_barrier();  // stage s is in LDS for everyone; stage s - 1 is consumed
    if (s + NS - 1 < total) issue_next(slot == 0 ? NS - 1 : slot - 1);
    mma_stage(ring + slot * G::kSlot, ring + G::kScaleBase + cg * G::kScales, cs);
    slot = slot == NS - 1 ? 0 : slot + 1;
    ++cs;
    if (cs % G::kGroup == 0 || (MB && cs == nst)) cg = cg == G::kBuffers - 1 ? 0 : cg + 1;
    if (MB && cs == nst) {
      epilogue(n0 + cb * FEAT);
      cs = 0;
      if (++cb < nb) zero_acc();
    }
  }
  if (!MB) epilogue(n0);
}

// ------------------------------------------------------------------ few rows

// A tile of at most 16 rows is a weight stream with little to multiply.  Its
// activation rows go to LDS whole, once per item, and every wave then streams
// weight rows of its own straight into registers, two chunks of kM4Steps
// steps in turn (the next one's loads in flight while one is multiplied):
// there is no barrier per stage, so no wave waits for another's loads, and
// LDS serves the activations only.  (Through the ring, whose stages all waves
// read at the same time, reads of activation tiles kept LDS busy for most of
// a stage: MI355X, 401 tokens, gate/up 4.5 TB/s.)
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
__device__ __forceinline__ bool m4_direct_fits(const Tile &t, int K) {
  return t.nrows <= kM4DirectRows && t.nrows * m4_direct_stride(K) <= kM4DirectAct;
}

// One chunk of a wave's two weight tiles of 16 rows.
struct M4Chunk {
  i32x4 raw[kM4Steps][2];
  uint32_t sc[2];  // lane group c: the scales of step c
};

// Output features [n0, n1) of a tile.
template <bool GATEUP>
__device__ __forceinline__ void m4_direct(const Mx4Args &a, const Tile &t, int n0, int n1,
                                          uint8_t *lds) {
  constexpr int FG = GATEUP ? 16 : 32;  // features of a wave's two weight tiles
  const int lane = lane_id();
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane >> 4, row = lane & 15;
  const int K = a.K, nk = K / 128;
  const int stride = m4_direct_stride(K);
  const int chunks = (nk + kM4Steps - 1) / kM4Steps;
  const int groups = max(((n1 - n0) / FG - wv + kM4Waves - 1) / kM4Waves, 0);
  const int total = groups * chunks;
  uint8_t *sc_lds = lds + kM4DirectAct + wv * kM4ScaleWave + row * kM4ScaleRow;

  auto load = [&](M4Chunk &q, int i) {
    const int g = i / chunks, s = (i - g * chunks) * kM4Steps;
    const int n = n0 + (wv + kM4Waves * g) * FG;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const size_t r = (size_t)t.e * a.N + n + row + (GATEUP ? 0 : 16 * w);
      const uint8_t *codes = (GATEUP && w ? a.w1 : a.w0) + r * (K / 2) + c * 16;
      const uint8_t *scales = (GATEUP && w ? a.s1 : a.s0) + r * (K / 32);
      // steps past the end load the last one again
      q.sc[w] = *reinterpret_cast<const uint32_t *>(scales + min(s + c, nk - 1) * 4);
#pragma unroll
      for (int u = 0; u < kM4Steps; ++u)
        q.raw[u][w] = *reinterpret_cast<const i32x4 *>(codes + min(s + u, nk - 1) * 64);
    }
    asm volatile("" ::: "memory");  // issued here, not where they are used
  };
  f32x4 acc[2] = {};
  const uint8_t *mine = lds + min(row, t.nrows - 1) * stride + c * 64;
  auto multiply = [&](const M4Chunk &q, int i) {
    const int g = i / chunks, ci = i - g * chunks, s = ci * kM4Steps;
    i32x4 ss[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      *reinterpret_cast<uint32_t *>(sc_lds + w * 16 * kM4ScaleRow + c * 4) = q.sc[w];
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
  if (total > 0) load(qa, 0);
  ring_barrier();  // every wave has read its item, which lies where the rows go
  // wave w brings rows w and w + 8
  for (int r = wv; r < t.nrows; r += kM4Waves) {
    const int i = t.row0 + r;
    const size_t s = GATEUP ? (size_t)(a.sorted_routes[i] / a.k) : (size_t)i;
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
  // no load in the loop is conditional: where a path without it joined, the
  // compiler would have to wait for all of them
  if (total == 0) return;
  int i = 0;
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

// ------------------------------------------------------------------ kernel

// The tile list, one thread per expert: its full 256-row tiles, then one
// remainder tile of the smallest capacity of 32, 64, 128, 192 and 256 rows
// that holds it (Tile); all tiles of a class together, tallest class first,
// experts in order.
constexpr int kM4ScheduleThreads = 256;  // the most experts
__global__ __launch_bounds__(kM4ScheduleThreads) void mx4_schedule_kernel(
    const int32_t *__restrict__ offsets, int E, M4Schedule *__restrict__ sch,
    Tile *__restrict__ tiles) {
  constexpr int NC = 5;  // capacities 256, 192, 128, 64, 32
  constexpr int NW = kM4ScheduleThreads / kWave;
  __shared__ int waves[NC][NW];
  const int e = threadIdx.x, lane = lane_id(), wave = threadIdx.x / kWave;
  int row0 = 0, n = 0;
  if (e < E) {
    row0 = offsets[e];
    n = offsets[e + 1] - row0;
  }
  const int full = n / kTileRows, rem = n % kTileRows;
  const int cls = rem == 0 ? NC : rem > 192 ? 0 : rem > 128 ? 1 : rem > 64 ? 2 : rem > 32 ? 3 : 4;
  int at[NC];  // where this expert's tiles of a class begin
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int mine = (c == 0 ? full : 0) + (c == cls ? 1 : 0);
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
  int total = 0, last = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    at[c] += total;
    last = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      if (w < wave) at[c] += waves[c][w];
      last += waves[c][w];
    }
    total += last;
  }
  const int only = n <= kTileRows ? kTileStream : 0;
  for (int i = 0; i < full; ++i) tiles[at[0] + i] = Tile{e, row0 + i * kTileRows, kTileRows, 8 | only};
  if (cls < NC) {
    constexpr int kAblk[NC] = {8, 6, 4, 2, 1};
    const int i = cls == 0 ? at[0] + full : cls == 1 ? at[1] : cls == 2 ? at[2] : cls == 3 ? at[3] : at[4];
    tiles[i] = Tile{e, row0 + full * kTileRows, rem, (cls == 0 ? kAblk[0] : cls == 1 ? kAblk[1] : cls == 2 ? kAblk[2] : cls == 3 ? kAblk[3] : kAblk[4]) | only};
  }
  if (e < 2 * kM4Queues) sch->heads[e / kM4Queues].head[e % kM4Queues] = 0;
  if (e < 2) sch->heads[e].left = 0;
  if (e == 0) {
    sch->n_tiles = total;
    sch->n_small = last;
  }
}

// Weight rows per item: 256; for 32-row tiles 128, in four blocks.
constexpr int kM4WRows = 256;
constexpr int kM4WRowsSmall = 128;

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
  __device__ __forceinline__ M4Queues(M4Heads *h_, int nbig_, int nsmall_, int ptb_, int pts_)
      : h(h_), nbig(nbig_), nsmall(nsmall_), ptb(ptb_), pts(pts_) {
    const int b = vreg((int)blockIdx.x);
    G = vreg((int)gridDim.x);
    q = b % kM4Queues;
    back = (b / kM4Queues) & 1;
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
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kM4Ring];
  // the next item (tile index, first feature; tile -1 = none left) is passed
  // from thread 0 through the idle ring between items
  int *next_item = reinterpret_cast<int *>(ring);
  const uint32_t ring_lds = lds_addr(ring);
  constexpr int kHalf = GATEUP ? 2 : 1;  // gate and up rows of one feature
  constexpr int FB = kM4WRows / kHalf;           // features per item of the taller tiles
  constexpr int FS = 4 * kM4WRowsSmall / kHalf;  // and of the 32-row tiles
  const int N = vreg(a.N);
  const int nsmall = vreg(*a.n_small), nbig = vreg(*a.ntiles) - nsmall;
  const int ptb = (N + FB - 1) / FB, pts = (N + FS - 1) / FS;  // items per tile
  M4Queues queues(a.heads, nbig, nsmall, ptb, pts);
  unsigned long long drawn = 0;
  bool begin = true;
  for (;;) {
    if (threadIdx.x == 0) {
      int ti = -1, part = 0;
      bool some = begin && queues.first(&ti, &part);
      if (begin && !some) drawn = queues.draw();
      if (!some) some = queues.take(drawn, &ti, &part);
      begin = false;
      next_item[0] = some ? ti : -1;
      next_item[1] = some ? part * (ti < nbig ? FB : FS) : 0;
      next_item[2] = a.K;
    }
    __syncthreads();
    // read before the item's first barrier (its loads overwrite it); the
    // reduction length comes through LDS so that nothing derived from it is
    // hoisted out of the loop into the scalar registers
    const int ti = __builtin_amdgcn_readfirstlane(next_item[0]);
    if (ti < 0) break;
    const int n0 = __builtin_amdgcn_readfirstlane(next_item[1]);
    Mx4Args ai = a;
    ai.K = __builtin_amdgcn_readfirstlane(next_item[2]);
    const Tile t = a.tiles[ti];
    if (threadIdx.x == 0) drawn = queues.draw();  // for the item after this one
    switch (tile_class(t)) {
      case 8: m4_item<GATEUP, false, 256, kM4WRows, 1>(ai, t, n0, 1, ring, ring_lds); break;
      case 6: m4_item<GATEUP, false, 192, kM4WRows, 1>(ai, t, n0, 1, ring, ring_lds); break;
      case 4: m4_item<GATEUP, false, 128, kM4WRows, 2>(ai, t, n0, 1, ring, ring_lds); break;
      case 2: m4_item<GATEUP, false, 64, kM4WRows, 2>(ai, t, n0, 1, ring, ring_lds); break;
      default: {
        const int n1 = min(n0 + FS, ai.N);
        const int nb = (n1 - n0) * 4 / FS;
        if (m4_direct_fits(t, ai.K))
          m4_direct<GATEUP>(ai, t, n0, n1, ring);
        else if (t.ablk & kTileStream)
          m4_item<GATEUP, true, 32, kM4WRowsSmall, 4>(ai, t, n0, nb, ring, ring_lds);
        else
          m4_item<GATEUP, false, 32, kM4WRowsSmall, 4>(ai, t, n0, nb, ring, ring_lds);
        break;
      }
    }
    // the ring (and the item in it) is rewritten only after every wave has
    // passed this barrier
    __syncthreads();
  }
}

hipError_t launch_ffn_mx4(const FfnLaunchMx4 &L, int stages, hipStream_t stream) {
  M4Schedule *sch = reinterpret_cast<M4Schedule *>(L.sch);
  if (stages & kStagePlan)
    hipLaunchKernelGGL(mx4_schedule_kernel, dim3(1), dim3(kM4ScheduleThreads), 0, stream, L.offsets,
                       L.E, sch, L.tiles);
  Mx4Args g{};
  g.k = L.k;
  g.tiles = L.tiles;
  g.ntiles = &sch->n_tiles;
  g.n_small = &sch->n_small;
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
    g.heads = &sch->heads[1];
    hipLaunchKernelGGL(grouped_gemm_mx4_kernel<false>, dim3(L.num_cus), dim3(kM4Threads), 0,
                       stream, g);
  }
  return hipGetLastError();
}

}  // namespace moe

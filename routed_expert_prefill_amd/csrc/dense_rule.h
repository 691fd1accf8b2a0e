// Which kernel an 8-bit product takes, from its sizes alone.  Host code without HIP, so
// that a test on the CPU can ask it too.
#pragma once

namespace moe {

// What a kernel of matmul_fp8.hip does with its sums: y = x w in bf16 or fp32,
// silu(x w) * (x w1) in fp32 or quantised by blocks, all through the bf16 instruction
// (short sums would have one code of h in five thousand fall the other way, and the
// layer's bf16 results 2.1e-3 to 2.6e-3 off in place of 1.7e-3); or y in bf16 with short
// sums, through the 8-bit one.
enum : int { kMmBf16, kMmF32, kMmSwiglu, kMmSwigluCodes, kMmShort, kMmModes };
constexpr bool mm_gateup(int mode) { return mode == kMmSwiglu || mode == kMmSwigluCodes; }

// The tiles to choose from, and the time of a round of them at 4096 columns (us,
// MI355X): `per` workgroups to each of 256 compute units.  Small tiles are bound by what
// a stage waits for (LDS, chained products), which several groups of waves shorten;
// large ones move less for each product.  By 4096 x 4096, bf16 results, in a graph:
//   100 rows   9.8 us in 32 x 64, 13.3 in 64 x 64, 14.0 in 32 x 32
//   401 rows   20.7 in 64 x 128, 23.5 two to a compute unit, 26 in 64 x 64, 34 in 32 x 64
//   2048 rows  60 in 128 x 256, 72 in 64 x 128 two to a compute unit, 82 one
//   8192 rows  238 in 128 x 256, 278 and 319 in 64 x 128
// and with short sums 401 rows 15.2 in 64 x 128, 8192 rows 130 in 256 x 256 (2.1 PFLOP/s),
// 155 in 128 x 256, 174 in 64 x 128.  The others would spill registers in tiles of
// 256 x 256; with codes converted again for every product they do not, and 8192 rows
// took 296 where 128 x 256 took 257.
//
// Rounds are taken to last in proportion to the columns.  At 128 and 256 columns, where
// a kernel's start is most of it, the tiles so chosen are up to 0.4 us slower than the
// best: 17 rows by 1024 x 128 4.2 us in 32 x 32 (seven of whose eight groups of waves
// have no block), 3.8 in 64 x 64; 33 by 4096 x 256 4.4 and 4.0; 300 by 2048 x 256 4.2 in
// 64 x 64, 5.2 in 64 x 128; 2048 by 4096 x 128 9.2 in 128 x 256, 10.1 in 64 x 128.
struct MmCost {
  int bm, bn;
  int per;                // workgroups to a compute unit in a full round
  float round[kMmModes];  // by what the kernel does; 0: not in these tiles
};
enum : int { k32x32, k32x64, k64x64, k64x128, k64x128Two, k64x256, k128x256, k256x256, kMmTiles };
constexpr MmCost kMmCosts[kMmTiles] = {
    {32, 32, 1, {5.9f, 5.9f, 0, 0, 5.6f}},
    {32, 64, 1, {8.0f, 8.0f, 8.0f, 0, 6.6f}},
    {64, 64, 1, {13.0f, 13.0f, 13.0f, 0, 9.4f}},
    {64, 128, 1, {20.0f, 20.0f, 20.0f, 0, 13.0f}},
    {64, 128, 2, {38.5f, 38.5f, 0, 0, 23.3f}},
    {64, 256, 1, {0, 0, 0, 38.0f, 0}},
    {128, 256, 1, {63.0f, 63.0f, 0, 66.0f, 37.5f}},
    {256, 256, 1, {0, 0, 0, 0, 69.5f}},
};
constexpr double kMmLaunch = 2.4;  // a launch more: rows, or h, quantised on their own

// The time of tiles i, beside what every kernel takes.
inline double mm_time(int i, int mode, int M, int N, int K) {
  const MmCost &c = kMmCosts[i];
  if (c.round[mode] == 0) return 1e30;
  const int bf = mm_gateup(mode) ? c.bn / 2 : c.bn;
  const double tiles = (double)((M - 1) / c.bm + 1) * ((N - 1) / bf + 1);
  double rounds = (double)(long long)((tiles - 1) / (256 * c.per)) + 1;
  if (c.per == 2 && tiles <= 256) rounds = 0.65;  // alone on its compute unit
  return rounds * c.round[mode] * K / 4096;
}

inline int mm_best(int mode, int M, int N, int K, double *time) {
  int best = -1;
  for (int i = 0; i < kMmTiles; ++i) {
    const double t = mm_time(i, mode, M, N, K);
    if (best < 0 || t < *time) {
      best = i;
      *time = t;
    }
  }
  return best;
}

// Whether gate and up write codes of h, in tiles that hold whole blocks of it.
inline bool gateup_quantises(int M, int N, int K) {
  double codes, h;
  mm_best(kMmSwigluCodes, M, N, K, &codes);
  mm_best(kMmSwiglu, M, N, K, &h);
  return codes < h + kMmLaunch;
}

// The kernel for few rows, matvec_fp8.hip: its rows, its columns of y (its workgroups
// lie in one line of fewer than 2^32 threads; times alone end below 2^18 columns), and
// the elements of x that each workgroup quantises by itself.
constexpr int kMatvecRows = 16;
constexpr int kMatvecCols = 1 << 20;
constexpr int kMatvecQuant = 8192;
inline bool matvec_quantises(int M, int K) {
  return M <= kMatvecRows && (long long)M * K <= kMatvecQuant;
}

// Whether it is the faster one; codes: x is quantised already.  A round of 256
// workgroups takes 3.1 us at 4096 columns and 0.12 more for each row (MI355X, us, in a
// graph): one row by 4096 5.0, in tiles of 32 x 32 6.8; 16 rows 7.3 and 7.0; by 16384
// one row 14.2, 16 rows 21.4, in tiles of 32 x 64 13.1.
inline bool product_is_matvec(int M, int N, int K, bool gateup, bool codes) {
  if (M > kMatvecRows || N > kMatvecCols) return false;
  double tiles;
  mm_best(gateup ? kMmSwiglu : kMmBf16, M, N, K, &tiles);
  const double groups = ((double)N - 1) / (gateup ? 8 : 16) + 1;
  double few = (3.1 + 0.12 * M) * ((double)(long long)((groups - 1) / 256) + 1) * K / 4096;
  if (!codes && !matvec_quantises(M, K)) few += kMmLaunch;
  if (!codes) tiles += kMmLaunch;
  return few <= tiles;
}

}  // namespace moe

// Launch entry points of the gfx950 kernels, called by the C ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"
#include "dense_rule.h"

namespace moe {

// Launches a kernel and returns the launch's own status.  (The thread's last
// error, which a launch in angle brackets leaves as the only sign, may be an
// earlier call's: the caller would then take a kernel that runs for one that
// does not.)
template <typename T>
struct LaunchArg {
  typedef T type;
};
template <typename... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t stream,
                  typename LaunchArg<P>::type... args) {
  void *ptrs[] = {const_cast<void *>(static_cast<const void *>(&args))...};
  const hipError_t err =
      hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, ptrs, 0, stream);
  if (err != hipSuccess) (void)hipGetLastError();  // reported here, not again by a later call
  return err;
}

hipError_t launch_route_build(const int32_t *ids, const uint8_t *mask, int R, int E,
                              int32_t *counts, int32_t *offsets, int32_t *sorted_routes,
                              int32_t *route_rows, int32_t *ws, hipStream_t stream);
size_t route_build_ws_bytes(int R, int E);

// The route build on the library's own device scratch (no workspace, no
// allocation), for up to kRouteNoAllocMaxR routes.
constexpr int kRouteNoAllocMaxR = 1 << 20;
hipError_t launch_route_build_noalloc(const int32_t *ids, const uint8_t *mask, int R, int E,
                                      int32_t *counts, int32_t *offsets, int32_t *sorted_routes,
                                      int32_t *route_rows, hipStream_t stream);

// row_limit (one int32: rows of y at or past it are never read), shared
// (fp32 [T,d]) and out_bf16 may be null; out may be null if out_bf16 is not.
hipError_t launch_combine(const float *y, const int32_t *route_rows, const float *topk_w,
                          const uint8_t *mask, const int32_t *row_limit, const float *shared,
                          int T, int k, int d, float *out, uint16_t *out_bf16,
                          hipStream_t stream);

hipError_t launch_route_topk(const float *logits, const float *bias, int T, int E, int k,
                             int32_t *ids, float *gates, int grid_cap, hipStream_t stream);

// Selection of experts from router scores (route_select.hip).
struct SelectArgs {
  const void *logits;  // [T, E] fp32, or bf16 without f32
  const float *bias;   // [E] or null
  int32_t *ids;        // [T, k]
  float *gates;        // [T, k]
  int T, E, k, groups, top_groups, group_top;
  float scale;
  bool f32, softmax, renormalise;
};
constexpr int kSelectMaxGroups = 64;
hipError_t launch_route_select(const SelectArgs &a, hipStream_t stream);

// E4M3 codes and scales of blocks of 128 elements (quant_blocks.hip).
hipError_t launch_quant_blocks(const void *x, bool f32, long long blocks, uint8_t *q, float *s,
                               hipStream_t stream);

// Product of E4M3 rows and weights with block scales (matmul_fp8.hip).  Columns
// are bounded so that 32-bit offsets reach the rows of a tile.
constexpr int kMatmulMaxK = 1 << 20;
struct MatmulArgs {
  const uint8_t *x;  // [M, K]
  const float *xs;   // [M, K / 128]
  const uint8_t *w;  // [N, K]
  const float *ws;   // [ceil(N / 128), K / 128]
  void *y;           // [M, N] fp32, or bf16 without f32
  int M, N, K;
  bool f32;
  bool short_sums;  // bf16 y through the 8-bit instruction
  // launch_gateup_fp8: the second matrix (w is gate, w1 up), and codes and scales of h
  const uint8_t *w1;
  const float *ws1;
  uint8_t *hq;  // [M, N]
  float *hs;    // [M, N / 128]
};
hipError_t launch_matmul_fp8(const MatmulArgs &a, hipStream_t stream);
// h = silu(x w) * (x w1): with gateup_quantises(M, N) codes and scales in hq and hs,
// otherwise fp32 in y.  N is a multiple of 128.
hipError_t launch_gateup_fp8(const MatmulArgs &a, hipStream_t stream);

// The same for at most kMatvecRows rows (matvec_fp8.hip).  With w1 and s1 (same
// sizes as w0, s0; N a multiple of 8): y = silu(x w0) * (x w1) in fp32.
struct MatvecArgs {
  const void *x;    // codes [M, K] with xs, else bf16 or (x_f32) fp32, quantised on the way
  const float *xs;  // [M, K / 128] or null, where matvec_quantises(M, K)
  const uint8_t *w0, *w1;
  const float *s0, *s1;
  void *y;  // [M, N] fp32, or bf16 without f32
  int M, N, K;
  bool x_f32, f32;
};
hipError_t launch_matvec_fp8(const MatvecArgs &a, hipStream_t stream);

int quant_max_cols();
hipError_t launch_quant_rows(const uint16_t *x, int rows, const int32_t *rows_dev, int cols,
                             uint8_t *q, float *s, int grid_cap, hipStream_t stream);

// Residual addition and root-mean-square norm of rows (norm.hip).
struct NormArgs {
  const void *x;         // [rows, d] bf16, or fp32 if x_f32
  const void *residual;  // [rows, d]; res_kind 0: none, 1: bf16, 2: fp32
  void *residual_out;    // as residual (as x without one), or null
  const void *weight;    // [d] bf16, or fp32 if w_f32
  uint16_t *y;           // bf16 [rows, d] or null
  uint8_t *q;            // E4M3 codes [rows, d] or null
  float *s;              // [rows], with q
  float eps;
  int rows, d;
  bool x_f32, w_f32;
  int res_kind;
};
int norm_max_cols();
hipError_t launch_add_rmsnorm(const NormArgs &a, hipStream_t stream);

// Tile list of the grouped FFN from the expert offsets (one thread per
// expert); also zeroes the work-queue heads.
hipError_t launch_grouped_schedule(const int32_t *offsets, int E, Schedule *sch, Tile *tiles,
                                   hipStream_t stream);

// Stages of the grouped FFN (bit mask).
enum : int { kStagePlan = 1, kStageGateUp = 2, kStageDown = 4, kStageAll = 7 };

// bf16 grouped FFN: schedule, gate/up + SwiGLU, down.
struct FfnLaunch {
  const uint16_t *x;
  const int32_t *offsets;
  const int32_t *sorted_routes;
  const uint16_t *wg, *wu, *wd;
  float *y;
  uint16_t *h;
  Schedule *sch;
  Tile *tiles;
  int T, k, E, d, f, R;
  int num_cus;  // workgroups of each persistent GEMM launch
};
hipError_t launch_grouped_ffn_bf16(const FfnLaunch &L, int stages, hipStream_t stream);

// fp8 grouped FFN: plan (schedule, per-row quantisation of x into qx, sx,
// row maxima of h cleared), gate/up + SwiGLU (h in bf16, its row maxima
// kept), down (per-row quantisation of h with those maxima, then GEMM).
struct FfnLaunchFp8 {
  const uint16_t *x;
  uint8_t *qx;
  float *sx;
  const int32_t *offsets;
  const int32_t *sorted_routes;
  const uint8_t *wg, *wu, *wd;
  const float *sg, *su, *sd;
  float *y;
  uint16_t *h;
  uint8_t *qh;
  float *sh;
  uint32_t *hmax;  // [R] bits of max |h| per row (the gate/up epilogue keeps them)
  Schedule *sch;
  Tile *tiles;
  int T, k, E, d, f, R;
  int grid_cap;  // workgroups of a row-quantisation launch
  int num_cus;
};
hipError_t launch_ffn_fp8(const FfnLaunchFp8 &L, int stages, hipStream_t stream);

// The widest rows of the MXFP4 kernels, whose loads take 32-bit offsets from a
// uniform base: 256 weight rows of codes to an item (2^31 bytes), and 128 rows of
// activations of a single-token call (2^31 elements).  Twice as wide would still
// do; at 2^26 columns the offsets, and the test for rows that fit LDS, wrap.
constexpr int kMx4MaxWidth = 1 << 24;

// Grouped FFN with MXFP4 weights and bf16 activations (ffn_mxfp4.hip).
struct FfnLaunchMx4 {
  const uint16_t *x;
  const int32_t *offsets;
  const int32_t *sorted_routes;
  const uint8_t *wg, *wu, *wd;  // codes, two to a byte
  const uint8_t *sg, *su, *sd;  // E8M0 scales
  float *y;
  uint16_t *h;
  Schedule *sch;
  Tile *tiles;
  int T, k, E, d, f, R;
  int num_cus;
};
hipError_t launch_ffn_mx4(const FfnLaunchMx4 &L, int stages, hipStream_t stream);

// Routed experts for single tokens, MXFP4 weights (decode_mxfp4.hip).
constexpr int kDecodeMaxRoutes = 64;
struct DecodeArgs {
  const uint16_t *x;    // [T, d]
  const int32_t *ids;   // [T, k]
  const float *w;       // [T, k]
  const uint8_t *mask;  // [T, k] or null
  const uint8_t *wg, *wu, *wd, *sg, *su, *sd;
  const float *shared;  // [T, d] or null
  uint16_t *h;          // [2, T * k, f]: the rounded values, then what that took
  float *out;           // [T, d] or null
  uint16_t *out_bf16;   // [T, d] or null
  int T, k, E, d, f, R;
};
hipError_t launch_decode_mx4(const DecodeArgs &a, hipStream_t stream);

// Per-row E4M3 quantisation of bf16 rows whose maxima are known: amax_bits[r]
// holds the fp32 bits of max |x[r, :]|; same codes and scales as
// launch_quant_rows.  rows_dev as there.
hipError_t launch_quant_rows_known_max(const uint16_t *x, int rows, const int32_t *rows_dev,
                                       int cols, const uint32_t *amax_bits, uint8_t *q, float *s,
                                       int grid_cap, hipStream_t stream);
// zero n 32-bit words (a kernel, not a memset: the path stays graph-capturable)
hipError_t launch_zero_u32(uint32_t *p, int n, hipStream_t stream);

}  // namespace moe

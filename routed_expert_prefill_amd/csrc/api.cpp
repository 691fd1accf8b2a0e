// Host side of the C ABI declared in include/moe_prefill.h: argument checks
// (all before any HIP call), workspace layout and launch sequencing.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "moe_prefill.h"
#include "kernels.h"


namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Scalars read once by a kernel (the combine's row limit) need only their
// own alignment.
bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

int status_from(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

int num_cus_current_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus <= 0)
    return 256;
  return cus;
}

// Workgroups of a row-quantisation launch: four per compute unit, each
// looping over rows.
int grid_cap_for_current_device() { return num_cus_current_device() * 4; }

struct FfnLayout {
  size_t sched, tiles, h, qx, sx, qh, sh, hmax, total;
};

bool ffn_desc_status(const moe_ffn_desc *d, int *st) {
  if (d == nullptr) {
    *st = MOE_EINVAL;
    return false;
  }
  if (d->T < 1 || d->k < 1 || d->E < 1 || d->d < 1 || d->f < 1) {
    *st = MOE_EINVAL;
    return false;
  }
  if ((long long)d->T * d->k >= (1LL << 31)) {
    *st = MOE_EINVAL;
    return false;
  }
  if (d->E > MOE_MAX_EXPERTS || d->k > MOE_MAX_TOPK || d->k > d->E || d->d % 128 != 0 ||
      d->f % 128 != 0) {
    *st = MOE_EUNSUPPORTED;
    return false;
  }
  const bool w8 = d->weight_dtype == MOE_W_FP8_E4M3_B128;
  const bool a8 = d->act_dtype == MOE_ACT_FP8_E4M3_ROW;
  const bool wok = d->weight_dtype == MOE_W_BF16 || d->weight_dtype == MOE_W_MXFP4 || w8;
  const bool aok = d->act_dtype == MOE_ACT_BF16 || a8;
  if (!wok || !aok || w8 != a8) {
    *st = MOE_EUNSUPPORTED;
    return false;
  }
  if (d->weight_dtype == MOE_W_MXFP4 && (d->d > moe::kMx4MaxWidth || d->f > moe::kMx4MaxWidth)) {
    *st = MOE_EUNSUPPORTED;
    return false;
  }
  if (a8 && (d->d > moe::quant_max_cols() || d->f > moe::quant_max_cols())) {
    *st = MOE_EUNSUPPORTED;
    return false;
  }
  *st = MOE_OK;
  return true;
}

// What moe_decode_ffn takes: MXFP4 weights and few routes.
int decode_desc_status(const moe_ffn_desc *d) {
  static_assert(MOE_DECODE_MAX_ROUTES == moe::kDecodeMaxRoutes, "one limit");
  int st;
  if (!ffn_desc_status(d, &st)) return st;
  if (d->weight_dtype != MOE_W_MXFP4 || d->T * d->k > MOE_DECODE_MAX_ROUTES)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

FfnLayout ffn_layout(const moe_ffn_desc *d) {
  const size_t R = (size_t)d->T * d->k;
  const bool fp8 = d->weight_dtype == MOE_W_FP8_E4M3_B128;
  FfnLayout L{};
  size_t off = 0;
  L.sched = off;
  off += align_up(sizeof(moe::Schedule));
  // at most R / 256 full tiles plus one remainder per expert (MXFP4: R / 64)
  const size_t full = d->weight_dtype == MOE_W_MXFP4 ? 64 : moe::kTileRows;
  L.tiles = off;
  off += align_up(sizeof(moe::Tile) * (R / full + (size_t)d->E));
  L.h = off;
  off += align_up(R * (size_t)d->f * 2);
  if (fp8) {
    L.qx = off;
    off += align_up((size_t)d->T * d->d);
    L.sx = off;
    off += align_up((size_t)d->T * 4);
    L.qh = off;
    off += align_up(R * (size_t)d->f);
    L.sh = off;
    off += align_up(R * 4);
    L.hmax = off;  // row maxima of |h|, kept by the gate/up epilogue
    off += align_up(R * 4);
  }
  L.total = off;
  return L;
}

}  // namespace

extern "C" {

const char *moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_EINVAL: return "MOE_EINVAL: invalid argument (null pointer, size or overflow)";
    case MOE_EUNSUPPORTED: return "MOE_EUNSUPPORTED: shape or dtype outside the supported set";
    case MOE_EALIGN: return "MOE_EALIGN: device pointer not 16-byte aligned";
    case MOE_EWORKSPACE: return "MOE_EWORKSPACE: workspace missing or too small";
    case MOE_EHIP: return "MOE_EHIP: HIP runtime error";
    case MOE_ETOOLARGE:
      return "MOE_ETOOLARGE: larger than the fixed device scratch of a no-allocation call";
    default: return "unknown moe_status";
  }
}

int moe_abi_version(void) { return 2; }

size_t moe_route_build_workspace(int T, int k, int E) {
  if (T < 1 || k < 1 || E < 1 || E > MOE_MAX_EXPERTS || (long long)T * k >= (1LL << 31)) return 0;
  return align_up(moe::route_build_ws_bytes(T * k, E));
}

int moe_route_build(const int32_t *topk_ids, const uint8_t *route_mask, int T, int k, int E,
                    int32_t *counts, int32_t *offsets, int32_t *sorted_routes,
                    int32_t *route_rows, void *workspace, size_t workspace_bytes,
                    moe_stream_t stream) {
  if (!topk_ids || !counts || !offsets || !sorted_routes || !route_rows) return MOE_EINVAL;
  if (T < 1 || k < 1 || (long long)T * k >= (1LL << 31)) return MOE_EINVAL;
  if (E < 1 || E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK || k > E) return MOE_EUNSUPPORTED;
  if (misaligned(topk_ids) || misaligned(counts) || misaligned(offsets) ||
      misaligned(sorted_routes) || misaligned(route_rows) || misaligned(workspace) ||
      (route_mask && misaligned(route_mask)))
    return MOE_EALIGN;
  const size_t need = moe_route_build_workspace(T, k, E);
  if (!workspace || workspace_bytes < need) return MOE_EWORKSPACE;
  return status_from(moe::launch_route_build(topk_ids, route_mask, T * k, E, counts, offsets,
                                             sorted_routes, route_rows,
                                             static_cast<int32_t *>(workspace),
                                             static_cast<hipStream_t>(stream)));
}

int moe_route_build_noalloc(const int32_t *topk_ids, const uint8_t *route_mask, int T, int k,
                            int E, int32_t *counts, int32_t *offsets, int32_t *sorted_routes,
                            int32_t *route_rows, moe_stream_t stream) {
  static_assert(MOE_ROUTE_NOALLOC_MAX_ROUTES == moe::kRouteNoAllocMaxR, "one limit");
  if (!topk_ids || !counts || !offsets || !sorted_routes || !route_rows) return MOE_EINVAL;
  if (T < 1 || k < 1 || (long long)T * k >= (1LL << 31)) return MOE_EINVAL;
  if (E < 1 || E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK || k > E) return MOE_EUNSUPPORTED;
  if ((long long)T * k > MOE_ROUTE_NOALLOC_MAX_ROUTES) return MOE_ETOOLARGE;
  if (misaligned(topk_ids) || misaligned(counts) || misaligned(offsets) ||
      misaligned(sorted_routes) || misaligned(route_rows) || (route_mask && misaligned(route_mask)))
    return MOE_EALIGN;
  return status_from(moe::launch_route_build_noalloc(topk_ids, route_mask, T * k, E, counts,
                                                     offsets, sorted_routes, route_rows,
                                                     static_cast<hipStream_t>(stream)));
}

size_t moe_grouped_ffn_workspace(const moe_ffn_desc *desc) {
  int st;
  if (!ffn_desc_status(desc, &st)) return 0;
  return ffn_layout(desc).total;
}

}  // extern "C"

namespace {

// The fp8 launch of a call whose arguments are checked, x quantised into the
// workspace.
moe::FfnLaunchFp8 fp8_launch(const moe_ffn_desc *desc, const void *x, const int32_t *offsets,
                             const int32_t *sorted_routes, const void *w_gate, const void *w_up,
                             const void *w_down, const void *s_gate, const void *s_up,
                             const void *s_down, float *y, char *ws) {
  const FfnLayout lay = ffn_layout(desc);
  moe::FfnLaunchFp8 L{};
  L.x = static_cast<const uint16_t *>(x);
  L.qx = reinterpret_cast<uint8_t *>(ws + lay.qx);
  L.sx = reinterpret_cast<float *>(ws + lay.sx);
  L.offsets = offsets;
  L.sorted_routes = sorted_routes;
  L.wg = static_cast<const uint8_t *>(w_gate);
  L.wu = static_cast<const uint8_t *>(w_up);
  L.wd = static_cast<const uint8_t *>(w_down);
  L.sg = static_cast<const float *>(s_gate);
  L.su = static_cast<const float *>(s_up);
  L.sd = static_cast<const float *>(s_down);
  L.y = y;
  L.h = reinterpret_cast<uint16_t *>(ws + lay.h);
  L.qh = reinterpret_cast<uint8_t *>(ws + lay.qh);
  L.sh = reinterpret_cast<float *>(ws + lay.sh);
  L.hmax = reinterpret_cast<uint32_t *>(ws + lay.hmax);
  L.sch = reinterpret_cast<moe::Schedule *>(ws + lay.sched);
  L.tiles = reinterpret_cast<moe::Tile *>(ws + lay.tiles);
  L.num_cus = num_cus_current_device();
  L.T = desc->T;
  L.k = desc->k;
  L.E = desc->E;
  L.d = desc->d;
  L.f = desc->f;
  L.R = desc->T * desc->k;
  L.grid_cap = grid_cap_for_current_device();
  return L;
}

// Shared body of moe_grouped_ffn and its stage calls.
int ffn_call(const moe_ffn_desc *desc, int stages, const void *x, const int32_t *offsets,
             const int32_t *sorted_routes, const void *w_gate, const void *w_up,
             const void *w_down, const void *s_gate, const void *s_up, const void *s_down,
             float *y, void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  int st;
  if (!ffn_desc_status(desc, &st)) return st;
  const bool fp8 = desc->weight_dtype == MOE_W_FP8_E4M3_B128;
  const bool mx4 = desc->weight_dtype == MOE_W_MXFP4;
  const bool scaled = fp8 || mx4;
  const bool plan = stages & moe::kStagePlan, gu = stages & moe::kStageGateUp,
             dn = stages & moe::kStageDown;
  // pointers each requested stage reads or writes
  if (plan && (!offsets || (fp8 && !x))) return MOE_EINVAL;
  if (gu && (!x || !sorted_routes || !w_gate || !w_up || (scaled && (!s_gate || !s_up))))
    return MOE_EINVAL;
  if (dn && (!offsets || !w_down || !y || (scaled && !s_down))) return MOE_EINVAL;
  const void *ptrs[] = {x, offsets, sorted_routes, w_gate, w_up, w_down, s_gate, s_up, s_down, y,
                        workspace};
  for (const void *p : ptrs)
    if (p && misaligned(p)) return MOE_EALIGN;
  const FfnLayout lay = ffn_layout(desc);
  if (!workspace || workspace_bytes < lay.total) return MOE_EWORKSPACE;

  char *ws = static_cast<char *>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int R = desc->T * desc->k;
  if (mx4) {
    moe::FfnLaunchMx4 L{};
    L.x = static_cast<const uint16_t *>(x);
    L.offsets = offsets;
    L.sorted_routes = sorted_routes;
    L.wg = static_cast<const uint8_t *>(w_gate);
    L.wu = static_cast<const uint8_t *>(w_up);
    L.wd = static_cast<const uint8_t *>(w_down);
    L.sg = static_cast<const uint8_t *>(s_gate);
    L.su = static_cast<const uint8_t *>(s_up);
    L.sd = static_cast<const uint8_t *>(s_down);
    L.y = y;
    L.h = reinterpret_cast<uint16_t *>(ws + lay.h);
    L.sch = reinterpret_cast<moe::Schedule *>(ws + lay.sched);
    L.tiles = reinterpret_cast<moe::Tile *>(ws + lay.tiles);
    L.num_cus = num_cus_current_device();
    L.T = desc->T;
    L.k = desc->k;
    L.E = desc->E;
    L.d = desc->d;
    L.f = desc->f;
    L.R = R;
    return status_from(moe::launch_ffn_mx4(L, stages, s));
  }
  if (!fp8) {
    moe::FfnLaunch L{};
    L.x = static_cast<const uint16_t *>(x);
    L.offsets = offsets;
    L.sorted_routes = sorted_routes;
    L.wg = static_cast<const uint16_t *>(w_gate);
    L.wu = static_cast<const uint16_t *>(w_up);
    L.wd = static_cast<const uint16_t *>(w_down);
    L.y = y;
    L.h = reinterpret_cast<uint16_t *>(ws + lay.h);
    L.sch = reinterpret_cast<moe::Schedule *>(ws + lay.sched);
    L.tiles = reinterpret_cast<moe::Tile *>(ws + lay.tiles);
    L.num_cus = num_cus_current_device();
    L.T = desc->T;
    L.k = desc->k;
    L.E = desc->E;
    L.d = desc->d;
    L.f = desc->f;
    L.R = R;
    return status_from(moe::launch_grouped_ffn_bf16(L, stages, s));
  }
  return status_from(moe::launch_ffn_fp8(
      fp8_launch(desc, x, offsets, sorted_routes, w_gate, w_up, w_down, s_gate, s_up, s_down, y, ws),
      stages, s));
}

}  // namespace

extern "C" {

int moe_grouped_ffn(const moe_ffn_desc *desc, const void *x, const int32_t *offsets,
                    const int32_t *sorted_routes, const void *w_gate, const void *w_up,
                    const void *w_down, const void *s_gate, const void *s_up,
                    const void *s_down, float *y, void *workspace, size_t workspace_bytes,
                    moe_stream_t stream) {
  return ffn_call(desc, moe::kStageAll, x, offsets, sorted_routes, w_gate, w_up, w_down, s_gate,
                  s_up, s_down, y, workspace, workspace_bytes, stream);
}

int moe_grouped_ffn_codes(const moe_ffn_desc *desc, const uint8_t *xq, const float *xs,
                          const int32_t *offsets, const int32_t *sorted_routes,
                          const void *w_gate, const void *w_up, const void *w_down,
                          const void *s_gate, const void *s_up, const void *s_down, float *y,
                          void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  int st;
  if (!ffn_desc_status(desc, &st)) return st;
  if (desc->weight_dtype != MOE_W_FP8_E4M3_B128) return MOE_EUNSUPPORTED;
  const void *ptrs[] = {xq,     xs,     offsets, sorted_routes, w_gate, w_up,
                        w_down, s_gate, s_up,    s_down,        y};
  for (const void *p : ptrs)
    if (!p) return MOE_EINVAL;
  for (const void *p : ptrs)
    if (misaligned(p)) return MOE_EALIGN;
  if (workspace && misaligned(workspace)) return MOE_EALIGN;
  if (!workspace || workspace_bytes < ffn_layout(desc).total) return MOE_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  moe::FfnLaunchFp8 L = fp8_launch(desc, nullptr, offsets, sorted_routes, w_gate, w_up, w_down,
                                   s_gate, s_up, s_down, y, static_cast<char *>(workspace));
  // read only: without the plan stage nothing writes the rows' codes
  L.qx = const_cast<uint8_t *>(xq);
  L.sx = const_cast<float *>(xs);
  // the plan without its quantisation
  hipError_t err = moe::launch_grouped_schedule(L.offsets, L.E, L.sch, L.tiles, s);
  if (err == hipSuccess) err = moe::launch_zero_u32(L.hmax, L.R, s);
  if (err == hipSuccess) err = moe::launch_ffn_fp8(L, moe::kStageGateUp | moe::kStageDown, s);
  return status_from(err);
}

int moe_ffn_plan(const moe_ffn_desc *desc, const void *x, const int32_t *offsets,
                 void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  return ffn_call(desc, moe::kStagePlan, x, offsets, nullptr, nullptr, nullptr, nullptr, nullptr,
                  nullptr, nullptr, nullptr, workspace, workspace_bytes, stream);
}

int moe_ffn_gate_up(const moe_ffn_desc *desc, const void *x, const int32_t *sorted_routes,
                    const void *w_gate, const void *w_up, const void *s_gate, const void *s_up,
                    void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  return ffn_call(desc, moe::kStageGateUp, x, nullptr, sorted_routes, w_gate, w_up, nullptr,
                  s_gate, s_up, nullptr, nullptr, workspace, workspace_bytes, stream);
}

int moe_ffn_down(const moe_ffn_desc *desc, const int32_t *offsets, const void *w_down,
                 const void *s_down, float *y, void *workspace, size_t workspace_bytes,
                 moe_stream_t stream) {
  return ffn_call(desc, moe::kStageDown, nullptr, offsets, nullptr, nullptr, nullptr, w_down,
                  nullptr, nullptr, s_down, y, workspace, workspace_bytes, stream);
}

int moe_combine(const float *y, const int32_t *route_rows, const float *topk_w,
                const uint8_t *route_mask, const int32_t *row_limit, int T, int k, int d,
                float *out, moe_stream_t stream) {
  if (!y || !route_rows || !topk_w || !out) return MOE_EINVAL;
  if (T < 1 || k < 1 || d < 4 || d % 4 != 0 || (long long)T * k >= (1LL << 31)) return MOE_EINVAL;
  if (k > MOE_MAX_TOPK) return MOE_EUNSUPPORTED;
  if (misaligned(y) || misaligned(route_rows) || misaligned(topk_w) || misaligned(out) ||
      (route_mask && misaligned(route_mask)) || (row_limit && misaligned4(row_limit)))
    return MOE_EALIGN;
  return status_from(moe::launch_combine(y, route_rows, topk_w, route_mask, row_limit, nullptr, T,
                                         k, d, out, nullptr, static_cast<hipStream_t>(stream)));
}

int moe_combine_shared(const float *y, const int32_t *route_rows, const float *topk_w,
                       const uint8_t *route_mask, const int32_t *row_limit, const float *shared,
                       int T, int k, int d, float *out, void *out_bf16, moe_stream_t stream) {
  if (!y || !route_rows || !topk_w || (!out && !out_bf16)) return MOE_EINVAL;
  if (T < 1 || k < 1 || d < 4 || d % 4 != 0 || (long long)T * k >= (1LL << 31)) return MOE_EINVAL;
  if (k > MOE_MAX_TOPK) return MOE_EUNSUPPORTED;
  const void *ptrs[] = {y, route_rows, topk_w, route_mask, shared, out, out_bf16};
  for (const void *p : ptrs)
    if (p && misaligned(p)) return MOE_EALIGN;
  if (row_limit && misaligned4(row_limit)) return MOE_EALIGN;
  return status_from(moe::launch_combine(y, route_rows, topk_w, route_mask, row_limit, shared, T,
                                         k, d, out, static_cast<uint16_t *>(out_bf16),
                                         static_cast<hipStream_t>(stream)));
}

int moe_route_topk(const float *logits, const float *bias, int T, int E, int k,
                   int32_t *topk_ids, float *topk_w, moe_stream_t stream) {
  if (!logits || !topk_ids || !topk_w) return MOE_EINVAL;
  if (T < 1 || E < 1 || k < 1 || (long long)T * E >= (1LL << 31)) return MOE_EINVAL;
  if (E > MOE_MAX_EXPERTS || k > MOE_MAX_TOPK || k > E) return MOE_EUNSUPPORTED;
  if (misaligned(logits) || misaligned(topk_ids) || misaligned(topk_w) || (bias && misaligned(bias)))
    return MOE_EALIGN;
  return status_from(moe::launch_route_topk(logits, bias, T, E, k, topk_ids, topk_w,
                                            num_cus_current_device() * 8,
                                            static_cast<hipStream_t>(stream)));
}

int moe_quant_rows_fp8(const void *x, int rows, int cols, uint8_t *q, float *s,
                       moe_stream_t stream) {
  if (!x || !q || !s || rows < 1 || cols < 1) return MOE_EINVAL;
  if (cols % 128 != 0 || cols > moe::quant_max_cols()) return MOE_EUNSUPPORTED;
  if (misaligned(x) || misaligned(q) || misaligned(s)) return MOE_EALIGN;
  return status_from(moe::launch_quant_rows(static_cast<const uint16_t *>(x), rows, nullptr, cols,
                                            q, s, grid_cap_for_current_device(),
                                            static_cast<hipStream_t>(stream)));
}

int moe_add_rmsnorm(const void *x, int x_dtype, const void *residual, void *residual_out,
                    int residual_dtype, const void *weight, int weight_dtype, float eps, int rows,
                    int d, void *y, uint8_t *q, float *s, moe_stream_t stream) {
  if (!x || !weight || (!y && !q) || (q == nullptr) != (s == nullptr)) return MOE_EINVAL;
  if (rows < 1 || d < 1 || !(eps > 0.0f) || !(eps < 3.40282347e38f)) return MOE_EINVAL;
  const auto known = [](int t) { return t == MOE_DT_BF16 || t == MOE_DT_F32; };
  if (!known(x_dtype) || !known(weight_dtype) || !known(residual_dtype)) return MOE_EUNSUPPORTED;
  if (!residual && residual_out && residual_dtype != x_dtype) return MOE_EUNSUPPORTED;
  if (d % 8 != 0 || d > moe::norm_max_cols()) return MOE_EUNSUPPORTED;
  const void *ptrs[] = {x, residual, residual_out, weight, y, q, s};
  for (const void *p : ptrs)
    if (p && misaligned(p)) return MOE_EALIGN;
  moe::NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.residual_out = residual_out;
  a.weight = weight;
  a.y = static_cast<uint16_t *>(y);
  a.q = q;
  a.s = s;
  a.eps = eps;
  a.rows = rows;
  a.d = d;
  a.x_f32 = x_dtype == MOE_DT_F32;
  a.w_f32 = weight_dtype == MOE_DT_F32;
  a.res_kind = !residual ? 0 : residual_dtype == MOE_DT_F32 ? 2 : 1;
  return status_from(moe::launch_add_rmsnorm(a, static_cast<hipStream_t>(stream)));
}

size_t moe_decode_ffn_workspace(const moe_ffn_desc *desc) {
  if (decode_desc_status(desc) != MOE_OK) return 0;
  return align_up((size_t)desc->T * desc->k * desc->f * 4);
}

int moe_decode_ffn(const moe_ffn_desc *desc, const void *x, const int32_t *topk_ids,
                   const float *topk_w, const uint8_t *route_mask, const void *w_gate,
                   const void *w_up, const void *w_down, const void *s_gate, const void *s_up,
                   const void *s_down, const float *shared, float *out, void *out_bf16,
                   void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  const int st = decode_desc_status(desc);
  if (st != MOE_OK) return st;
  if (!x || !topk_ids || !topk_w || !w_gate || !w_up || !w_down || !s_gate || !s_up || !s_down ||
      (!out && !out_bf16))
    return MOE_EINVAL;
  const void *ptrs[] = {x,     topk_ids, topk_w, route_mask, w_gate, w_up,     w_down,
                        s_gate, s_up,    s_down, shared,     out,    out_bf16, workspace};
  for (const void *p : ptrs)
    if (p && misaligned(p)) return MOE_EALIGN;
  if (!workspace || workspace_bytes < moe_decode_ffn_workspace(desc)) return MOE_EWORKSPACE;
  moe::DecodeArgs a{};
  a.x = static_cast<const uint16_t *>(x);
  a.ids = topk_ids;
  a.w = topk_w;
  a.mask = route_mask;
  a.wg = static_cast<const uint8_t *>(w_gate);
  a.wu = static_cast<const uint8_t *>(w_up);
  a.wd = static_cast<const uint8_t *>(w_down);
  a.sg = static_cast<const uint8_t *>(s_gate);
  a.su = static_cast<const uint8_t *>(s_up);
  a.sd = static_cast<const uint8_t *>(s_down);
  a.shared = shared;
  a.h = static_cast<uint16_t *>(workspace);
  a.out = out;
  a.out_bf16 = static_cast<uint16_t *>(out_bf16);
  a.T = desc->T;
  a.k = desc->k;
  a.E = desc->E;
  a.d = desc->d;
  a.f = desc->f;
  a.R = desc->T * desc->k;
  return status_from(moe::launch_decode_mx4(a, static_cast<hipStream_t>(stream)));
}

int moe_route_select(const moe_select_desc *desc, const void *logits, const float *bias,
                     int32_t *topk_ids, float *topk_w, moe_stream_t stream) {
  if (!desc || !logits || !topk_ids || !topk_w) return MOE_EINVAL;
  const moe_select_desc &d = *desc;
  if (d.T < 1 || d.E < 1 || d.k < 1 || d.groups < 1 || d.top_groups < 1 ||
      (long long)d.T * d.E >= (1LL << 31) || !std::isfinite(d.scale))
    return MOE_EINVAL;
  const bool types = (d.logits_dtype == MOE_DT_BF16 || d.logits_dtype == MOE_DT_F32) &&
                     (d.scores == MOE_SCORES_SOFTMAX || d.scores == MOE_SCORES_SIGMOID);
  if (!types || d.E > MOE_MAX_EXPERTS || d.k > MOE_MAX_TOPK || d.groups > moe::kSelectMaxGroups ||
      d.E % d.groups != 0 || d.top_groups > d.groups || d.k > d.top_groups * (d.E / d.groups) ||
      (d.group_top != 1 && d.group_top != 2))
    return MOE_EUNSUPPORTED;
  if (misaligned(logits) || misaligned(topk_ids) || misaligned(topk_w) || (bias && misaligned(bias)))
    return MOE_EALIGN;
  moe::SelectArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.gates = topk_w;
  a.T = d.T;
  a.E = d.E;
  a.k = d.k;
  a.groups = d.groups;
  a.top_groups = d.top_groups;
  a.group_top = d.group_top;
  a.scale = d.scale;
  a.f32 = d.logits_dtype == MOE_DT_F32;
  a.softmax = d.scores == MOE_SCORES_SOFTMAX;
  a.renormalise = d.renormalise != 0;
  return status_from(moe::launch_route_select(a, static_cast<hipStream_t>(stream)));
}

int moe_quant_blocks_fp8(const void *x, int x_dtype, int rows, int cols, uint8_t *q, float *s,
                         moe_stream_t stream) {
  if (!x || !q || !s || rows < 1 || cols < 1) return MOE_EINVAL;
  if ((x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_F32) || cols % 128 != 0) return MOE_EUNSUPPORTED;
  if (misaligned(x) || misaligned(q) || misaligned(s)) return MOE_EALIGN;
  const long long blocks = (long long)rows * (cols / 128);
  return status_from(moe::launch_quant_blocks(x, x_dtype == MOE_DT_F32, blocks, q, s,
                                              static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

int matmul_status(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1) return MOE_EINVAL;
  // a workgroup to 32 rows by 32 columns at the least, fewer than 2^31 of them
  const long long most = (((long long)M + 31) / 32) * (((long long)N + 31) / 32);
  if (K % 128 != 0 || K > moe::kMatmulMaxK || most >= (1LL << 31)) return MOE_EUNSUPPORTED;
  // a tile's rows and columns are counted in 32 bits
  if (M > INT32_MAX - 256 || N > INT32_MAX - 256) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// Codes and scales of M rows of K columns, from offset `at` on.
struct CodesLayout {
  size_t q, s, end;
};
CodesLayout codes_layout(size_t at, int M, int K) {
  CodesLayout L{};
  L.q = at;
  L.s = L.q + align_up((size_t)M * K);
  L.end = L.s + align_up((size_t)M * (K / 128) * 4);
  return L;
}

struct SharedLayout {
  CodesLayout x, h;
  size_t hf, total;  // h in fp32
};
SharedLayout shared_layout(int T, int d, int f) {
  SharedLayout L{};
  L.x = codes_layout(0, T, d);
  L.h = codes_layout(L.x.end, T, f);
  L.hf = L.h.end;
  L.total = L.hf + align_up((size_t)T * f * 4);
  return L;
}

int shared_status(int T, int d, int f) {
  if (T < 1 || d < 1 || f < 1) return MOE_EINVAL;
  if (d % 128 != 0 || f % 128 != 0) return MOE_EUNSUPPORTED;
  const int st = matmul_status(T, f, d);
  return st != MOE_OK ? st : matmul_status(T, d, f);
}

// A product of a call whose arguments are checked; without xs x is bf16, or fp32
// with x_f32, and is quantised into `codes` (K columns' layout at `room`) where the
// kernel does not do so itself.
struct Product {
  const void *x;
  const float *xs;
  bool x_f32;
  int M, N, K;
  char *room;
  CodesLayout codes;
};

hipError_t quantise(Product *p, hipStream_t s) {
  uint8_t *q = reinterpret_cast<uint8_t *>(p->room + p->codes.q);
  float *scales = reinterpret_cast<float *>(p->room + p->codes.s);
  const hipError_t err = moe::launch_quant_blocks(p->x, p->x_f32, (long long)p->M * (p->K / 128), q,
                                                  scales, s);
  p->x = q;
  p->xs = scales;
  return err;
}

moe::MatmulArgs matmul_args(const Product &p, const uint8_t *w, const float *ws) {
  moe::MatmulArgs a{};
  a.x = static_cast<const uint8_t *>(p.x);
  a.xs = p.xs;
  a.w = w;
  a.ws = ws;
  a.M = p.M;
  a.N = p.N;
  a.K = p.K;
  return a;
}

moe::MatvecArgs matvec_args(const Product &p, const uint8_t *w, const float *ws, void *y,
                            bool f32) {
  moe::MatvecArgs a{};
  a.x = p.x;
  a.xs = p.xs;
  a.w0 = w;
  a.s0 = ws;
  a.y = y;
  a.M = p.M;
  a.N = p.N;
  a.K = p.K;
  a.x_f32 = p.x_f32;
  a.f32 = f32;
  return a;
}

// A result's type with its flag; false where there is no such.
struct Result {
  bool f32, short_sums;
};
bool result_type(int y_dtype, Result *r) {
  r->f32 = y_dtype == MOE_DT_F32;
  r->short_sums = y_dtype == (MOE_DT_BF16 | MOE_SHORT_SUMS);
  return r->f32 || r->short_sums || y_dtype == MOE_DT_BF16;
}

// y = x w
hipError_t product(Product p, const uint8_t *w, const float *ws, void *y, Result r, hipStream_t s) {
  const bool few = moe::product_is_matvec(p.M, p.N, p.K, false, p.xs != nullptr);
  hipError_t err = hipSuccess;
  if (!p.xs && !(few && moe::matvec_quantises(p.M, p.K))) err = quantise(&p, s);
  if (err != hipSuccess) return err;
  if (few) return moe::launch_matvec_fp8(matvec_args(p, w, ws, y, r.f32), s);
  moe::MatmulArgs a = matmul_args(p, w, ws);
  a.y = y;
  a.f32 = r.f32;
  a.short_sums = r.short_sums;
  return moe::launch_matmul_fp8(a, s);
}

// down's rows = silu(x w0) * (x w1), in fp32 in h or as codes in down's room.
hipError_t gate_up(Product p, const uint8_t *w0, const float *s0, const uint8_t *w1,
                   const float *s1, float *h, Product *down, hipStream_t s) {
  const bool few = moe::product_is_matvec(p.M, p.N, p.K, true, p.xs != nullptr);
  hipError_t err = hipSuccess;
  if (!p.xs && !(few && moe::matvec_quantises(p.M, p.K))) err = quantise(&p, s);
  if (err != hipSuccess) return err;
  down->x = h;
  down->xs = nullptr;
  down->x_f32 = true;
  if (few) {
    moe::MatvecArgs a = matvec_args(p, w0, s0, h, true);
    a.w1 = w1;
    a.s1 = s1;
    return moe::launch_matvec_fp8(a, s);
  }
  moe::MatmulArgs a = matmul_args(p, w0, s0);
  a.w1 = w1;
  a.ws1 = s1;
  if (moe::gateup_quantises(p.M, p.N, p.K)) {
    a.hq = reinterpret_cast<uint8_t *>(down->room + down->codes.q);
    a.hs = reinterpret_cast<float *>(down->room + down->codes.s);
    down->x = a.hq;
    down->xs = a.hs;
  } else {
    a.y = h;
  }
  return moe::launch_gateup_fp8(a, s);
}

}  // namespace

extern "C" {

size_t moe_matmul_fp8_workspace(int M, int N, int K) {
  return matmul_status(M, N, K) == MOE_OK ? codes_layout(0, M, K).end : 0;
}

int moe_matmul_fp8(const void *x, const float *xs, int M, int N, int K, const uint8_t *w,
                   const float *ws, void *y, int y_dtype, void *workspace, size_t workspace_bytes,
                   moe_stream_t stream) {
  if (!x || !w || !ws || !y) return MOE_EINVAL;
  const int st = matmul_status(M, N, K);
  if (st != MOE_OK) return st;
  Result type;
  if (!result_type(y_dtype, &type)) return MOE_EUNSUPPORTED;
  const void *ptrs[] = {x, xs, w, ws, y, workspace};
  for (const void *p : ptrs)
    if (p && misaligned(p)) return MOE_EALIGN;
  const CodesLayout L = codes_layout(0, M, K);
  if (!xs && (!workspace || workspace_bytes < L.end)) return MOE_EWORKSPACE;
  const Product p = {x, xs, false, M, N, K, static_cast<char *>(workspace), L};
  return status_from(product(p, w, ws, y, type, static_cast<hipStream_t>(stream)));
}

size_t moe_shared_ffn_workspace(int T, int d, int f) {
  return shared_status(T, d, f) == MOE_OK ? shared_layout(T, d, f).total : 0;
}

int moe_shared_ffn(const void *x, const float *xs, int T, int d, int f, const uint8_t *w_gate,
                   const uint8_t *w_up, const uint8_t *w_down, const float *s_gate,
                   const float *s_up, const float *s_down, void *out, int out_dtype,
                   void *workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!x || !w_gate || !w_up || !w_down || !s_gate || !s_up || !s_down || !out) return MOE_EINVAL;
  const int st = shared_status(T, d, f);
  if (st != MOE_OK) return st;
  Result type;
  if (!result_type(out_dtype, &type)) return MOE_EUNSUPPORTED;
  const void *ptrs[] = {x, xs, w_gate, w_up, w_down, s_gate, s_up, s_down, out, workspace};
  for (const void *p : ptrs)
    if (p && misaligned(p)) return MOE_EALIGN;
  const SharedLayout L = shared_layout(T, d, f);
  if (!workspace || workspace_bytes < L.total) return MOE_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char *base = static_cast<char *>(workspace);
  const Product up = {x, xs, false, T, f, d, base, L.x};
  Product down = {nullptr, nullptr, true, T, d, f, base, L.h};
  hipError_t err = gate_up(up, w_gate, s_gate, w_up, s_up, reinterpret_cast<float *>(base + L.hf),
                           &down, s);
  if (err == hipSuccess) err = product(down, w_down, s_down, out, type, s);
  return status_from(err);
}

}  // extern "C"

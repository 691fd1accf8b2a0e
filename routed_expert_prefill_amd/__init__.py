"""Grouped routed-MoE prefill on gfx950: Python binding of the C ABI.

The three calls mirror include/moe_prefill.h one to one; every step runs in
the HIP library.  This module only checks tensor placement/dtypes, passes raw
device pointers and the current HIP stream, and allocates outputs and
workspaces with torch.  There is no CPU fallback: if the library is missing,
every call raises.
"""
from __future__ import annotations

import ctypes
import operator
from typing import NamedTuple, Optional

from . import _lib
from ._lib import (MOE_ACT_BF16, MOE_ACT_FP8_E4M3_ROW, MOE_W_BF16, MOE_W_FP8_E4M3_B128,
                   MOE_SCORES_SIGMOID, MOE_SCORES_SOFTMAX, MOE_SHORT_SUMS, MOE_W_MXFP4,
                   LibraryNotBuilt, MoeFfnDesc)

__all__ = [
    "route_topk", "route_build", "route_build_noalloc", "grouped_ffn", "grouped_ffn_codes", "combine", "combine_shared", "quant_rows_fp8", "add_rmsnorm", "decode_ffn", "route_select", "quant_blocks_fp8", "matmul_fp8", "shared_ffn", "MoEPrefill", "RouteTable",
    "ffn_desc", "ffn_plan", "ffn_gate_up", "ffn_down", "LibraryNotBuilt", "load_library",
]


def load_library():
    return _lib.load()


class RouteTable(NamedTuple):
    counts: "torch.Tensor"  # int32 [E+1]
    offsets: "torch.Tensor"  # int32 [E+2]
    sorted_routes: "torch.Tensor"  # int32 [T*k]
    route_rows: "torch.Tensor"  # int32 [T*k]


_torch_module = None


def _torch():
    # imported with the first call, and kept: the import statement alone is
    # 0.3 us, several times a call
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


_native_module = False


def _native():
    """The extension module of csrc/binding.cpp, bound to the loaded library,
    or None where it is not built: the calls then go the way of the others."""
    global _native_module
    if _native_module is False:
        lib = _lib.load()
        _torch()  # whose libraries the module needs loaded
        try:
            from . import _binding
        except ImportError:
            _binding = None
        else:
            _binding.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                            for f in (lib.moe_add_rmsnorm, lib.moe_decode_ffn)))
            _binding.bind_dense(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.moe_route_select, lib.moe_quant_blocks_fp8, lib.moe_matmul_fp8_workspace,
                lib.moe_matmul_fp8, lib.moe_shared_ffn_workspace, lib.moe_shared_ffn)))
        _native_module = _binding
    return _native_module


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    # the raw handle of torch.cuda.current_stream(), without making a Stream
    # object for it (about 3 us a call)
    C = _torch()._C
    return C._cuda_getCurrentRawStream(C._cuda_getDevice())


def _need(t, name, dtype, ndim=None):
    try:
        if (t.is_cuda and t.dtype == (dtype or t.dtype) and (ndim is None or t.dim() == ndim)
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def route_topk(logits, k: int, bias=None, topk_ids=None, topk_w=None):
    """moe_route_topk: top-k experts (descending, ties to the lower index) and
    renormalised gates from fp32 router logits [T, E]."""
    torch = _torch()
    lib = _lib.load()
    _need(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    if bias is not None:
        _need(bias, "bias", torch.float32, 1)
        if bias.numel() != E:
            raise ValueError("bias must have E entries")
    if topk_ids is None:
        topk_ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty(T, k, dtype=torch.float32, device=logits.device)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_w, "topk_w", torch.float32, 2)
    rc = lib.moe_route_topk(_ptr(logits), _ptr(bias), T, E, k, _ptr(topk_ids), _ptr(topk_w),
                            _stream())
    _lib.check(rc, "moe_route_topk")
    return topk_ids, topk_w


def route_build(topk_ids, route_mask, E: int, out: Optional[RouteTable] = None,
                workspace=None) -> RouteTable:
    """moe_route_build: histogram, prefix and stable scatter of the routes."""
    torch = _torch()
    lib = _lib.load()
    _need(topk_ids, "topk_ids", torch.int32, 2)
    if route_mask is not None:
        _need(route_mask, "route_mask", torch.uint8, 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    if out is None:
        out = RouteTable(
            counts=torch.empty(E + 1, dtype=torch.int32, device=dev),
            offsets=torch.empty(E + 2, dtype=torch.int32, device=dev),
            sorted_routes=torch.empty(T * k, dtype=torch.int32, device=dev),
            route_rows=torch.empty(T * k, dtype=torch.int32, device=dev),
        )
    if workspace is None:
        wsb = lib.moe_route_build_workspace(T, k, E)
        workspace = torch.empty(max(wsb, 256), dtype=torch.uint8, device=dev)
    rc = lib.moe_route_build(_ptr(topk_ids), _ptr(route_mask), T, k, E, _ptr(out.counts),
                             _ptr(out.offsets), _ptr(out.sorted_routes), _ptr(out.route_rows),
                             _ptr(workspace), workspace.numel(), _stream())
    _lib.check(rc, "moe_route_build")
    return out


def route_build_noalloc(topk_ids, route_mask, E: int, out: Optional[RouteTable] = None) -> RouteTable:
    """moe_route_build_noalloc: the route build on the library's own device
    scratch (no workspace); at most MOE_ROUTE_NOALLOC_MAX_ROUTES routes.  The
    outputs are allocated here unless given; the C call allocates nothing."""
    torch = _torch()
    lib = _lib.load()
    _need(topk_ids, "topk_ids", torch.int32, 2)
    if route_mask is not None:
        _need(route_mask, "route_mask", torch.uint8, 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    if out is None:
        out = RouteTable(
            counts=torch.empty(E + 1, dtype=torch.int32, device=dev),
            offsets=torch.empty(E + 2, dtype=torch.int32, device=dev),
            sorted_routes=torch.empty(T * k, dtype=torch.int32, device=dev),
            route_rows=torch.empty(T * k, dtype=torch.int32, device=dev),
        )
    rc = lib.moe_route_build_noalloc(_ptr(topk_ids), _ptr(route_mask), T, k, E, _ptr(out.counts),
                                     _ptr(out.offsets), _ptr(out.sorted_routes),
                                     _ptr(out.route_rows), _stream())
    _lib.check(rc, "moe_route_build_noalloc")
    return out


def ffn_desc(T: int, k: int, E: int, d: int, f: int, fp8: bool = False,
             weights: Optional[str] = None) -> MoeFfnDesc:
    """Shapes and formats of a layer; weights: "bf16", "fp8" or "mxfp4"
    (default: by fp8)."""
    if weights is None:
        weights = "fp8" if fp8 else "bf16"
    if weights not in _WEIGHTS:
        raise ValueError(f"weights must be one of {sorted(_WEIGHTS)}, got {weights!r}")
    if fp8 and weights != "fp8":
        raise ValueError(f"fp8=True contradicts weights={weights!r}")
    return MoeFfnDesc(T, k, E, d, f, *_WEIGHTS[weights])


# weight and activation formats by name
_WEIGHTS = {"bf16": (MOE_W_BF16, MOE_ACT_BF16),
            "fp8": (MOE_W_FP8_E4M3_B128, MOE_ACT_FP8_E4M3_ROW),
            "mxfp4": (MOE_W_MXFP4, MOE_ACT_BF16)}


def _need_mx4(x, offsets, sorted_routes, E, f, w_gate, w_up, w_down, s_gate, s_up, s_down):
    """Codes and scales of MXFP4 weights: [E, rows, cols/2] and [E, rows, cols/32];
    everything on the device of x, the current one."""
    u8, d = (_torch().uint8,), x.shape[1]
    dev = _on_current(x, "x")
    for name, w, s, rows, cols in (("gate", w_gate, s_gate, f, d), ("up", w_up, s_up, f, d),
                                   ("down", w_down, s_down, d, f)):
        _need_rows(w, "w_" + name, (E, rows, cols // 2), u8, dev)
        _need_rows(s, "s_" + name, (E, rows, cols // 32), u8, dev)
    for name, t in (("offsets", offsets), ("sorted_routes", sorted_routes)):
        _need_rows(t, name, t.shape, (t.dtype,), dev)


def _need_y(y, R, d, workspace, device):
    """y for R sorted rows, or more, and the workspace beside it."""
    torch = _torch()
    _need(y, "y", torch.float32, 2)
    _need_rows(y, "y", (max(R, y.shape[0]), d), (torch.float32,), device)
    _need_rows(workspace, "workspace", workspace.shape, (torch.uint8,), device)


def grouped_ffn(x, offsets, sorted_routes, w_gate, w_up, w_down, k: int, s_gate=None,
                s_up=None, s_down=None, y=None, workspace=None):
    """moe_grouped_ffn: y[i] = Wd . bf16(silu(Wg . x) * (Wu . x)) per sorted row i.

    Weights bf16; E4M3 codes (uint8) with fp32 block scales; or MXFP4 codes
    (uint8, two columns to a byte) with E8M0 scales (uint8, one for 32 columns
    of a row)."""
    torch = _torch()
    lib = _lib.load()
    mx4 = w_gate.dtype == torch.uint8 and s_gate is not None and s_gate.dtype == torch.uint8
    fp8 = w_gate.dtype == torch.uint8 and not mx4
    _need(x, "x", torch.bfloat16, 2)
    wdt = torch.uint8 if fp8 or mx4 else torch.bfloat16
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(w, name, wdt, 3)
    _need(offsets, "offsets", torch.int32, 1)
    _need(sorted_routes, "sorted_routes", torch.int32, 1)
    if fp8:
        for name, s in (("s_gate", s_gate), ("s_up", s_up), ("s_down", s_down)):
            _need(s, name, torch.float32, 3)
    T, d = x.shape
    E, f, d2 = w_gate.shape
    if mx4:
        _need_mx4(x, offsets, sorted_routes, E, f, w_gate, w_up, w_down, s_gate, s_up, s_down)
    elif d2 != d or tuple(w_up.shape) != (E, f, d) or tuple(w_down.shape) != (E, d, f):
        raise ValueError("weight shapes must be w_gate/w_up [E,f,d] and w_down [E,d,f]")
    if offsets.numel() != E + 2 or sorted_routes.numel() != T * k:
        raise ValueError("offsets must have E+2 entries and sorted_routes T*k")
    desc = ffn_desc(T, k, E, d, f, weights="mxfp4" if mx4 else "fp8" if fp8 else "bf16")
    if y is None:
        y = torch.empty(T * k, d, dtype=torch.float32, device=x.device)
    _need(y, "y", torch.float32, 2)
    if workspace is None:
        workspace = _ffn_ws(desc, x.device, None)
    if mx4:
        _need_y(y, T * k, d, workspace, x.device)
    rc = lib.moe_grouped_ffn(ctypes.byref(desc), _ptr(x), _ptr(offsets), _ptr(sorted_routes),
                             _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(s_gate), _ptr(s_up),
                             _ptr(s_down), _ptr(y), _ptr(workspace), workspace.numel(), _stream())
    _lib.check(rc, "moe_grouped_ffn")
    return y


def grouped_ffn_codes(xq, xs, offsets, sorted_routes, w_gate, w_up, w_down, k: int, s_gate, s_up,
                      s_down, y=None, workspace=None):
    """moe_grouped_ffn_codes: the fp8 grouped_ffn on rows that are quantised
    already -- E4M3 codes xq (uint8) [T, d] and scales xs [T], as add_rmsnorm
    and quant_rows_fp8 give them."""
    torch = _torch()
    lib = _lib.load()
    dev = _on_current(xq, "xq")
    _need(xq, "xq", torch.uint8, 2)
    _need(w_gate, "w_gate", torch.uint8, 3)
    T, d = xq.shape
    E, f, _ = w_gate.shape
    u8, f32, i32 = (torch.uint8,), (torch.float32,), (torch.int32,)
    for name, t, shape, dtypes in (
            ("xs", xs, (T,), f32), ("w_gate", w_gate, (E, f, d), u8), ("w_up", w_up, (E, f, d), u8),
            ("w_down", w_down, (E, d, f), u8), ("s_gate", s_gate, (E, f // 128, d // 128), f32),
            ("s_up", s_up, (E, f // 128, d // 128), f32),
            ("s_down", s_down, (E, d // 128, f // 128), f32), ("offsets", offsets, (E + 2,), i32),
            ("sorted_routes", sorted_routes, (T * k,), i32)):
        _need_rows(t, name, shape, dtypes, dev)
    desc = ffn_desc(T, k, E, d, f, weights="fp8")
    if y is None:
        y = torch.empty(T * k, d, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = _ffn_ws(desc, dev, None)
    _need_y(y, T * k, d, workspace, dev)
    rc = lib.moe_grouped_ffn_codes(ctypes.byref(desc), _ptr(xq), _ptr(xs), _ptr(offsets),
                                   _ptr(sorted_routes), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                   _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(y),
                                   _ptr(workspace), workspace.numel(), _stream())
    _lib.check(rc, "moe_grouped_ffn_codes")
    return y


def _ffn_ws(desc, device, workspace):
    torch = _torch()
    lib = _lib.load()
    need = lib.moe_grouped_ffn_workspace(ctypes.byref(desc))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return workspace


def ffn_plan(desc: MoeFfnDesc, x, offsets, workspace):
    """moe_ffn_plan: tile schedule from offsets (fp8: also quantises x)."""
    lib = _lib.load()
    rc = lib.moe_ffn_plan(ctypes.byref(desc), _ptr(x), _ptr(offsets), _ptr(workspace),
                          workspace.numel(), _stream())
    _lib.check(rc, "moe_ffn_plan")


def ffn_gate_up(desc: MoeFfnDesc, x, sorted_routes, w_gate, w_up, s_gate, s_up, workspace):
    """moe_ffn_gate_up: gate/up GEMM with the SwiGLU epilogue, h into the workspace."""
    lib = _lib.load()
    rc = lib.moe_ffn_gate_up(ctypes.byref(desc), _ptr(x), _ptr(sorted_routes), _ptr(w_gate),
                             _ptr(w_up), _ptr(s_gate), _ptr(s_up), _ptr(workspace),
                             workspace.numel(), _stream())
    _lib.check(rc, "moe_ffn_gate_up")


def ffn_down(desc: MoeFfnDesc, offsets, w_down, s_down, y, workspace):
    """moe_ffn_down: (fp8: per-row quantisation of h) down GEMM into y."""
    lib = _lib.load()
    rc = lib.moe_ffn_down(ctypes.byref(desc), _ptr(offsets), _ptr(w_down), _ptr(s_down), _ptr(y),
                          _ptr(workspace), workspace.numel(), _stream())
    _lib.check(rc, "moe_ffn_down")


def _row_limit(row_limit):
    """The combine's row bound: a one-element int32 device tensor (for
    instance ``offsets[E:E + 1]`` of a route table) or None."""
    torch = _torch()
    if row_limit is None:
        return None
    if not isinstance(row_limit, torch.Tensor) or row_limit.dtype != torch.int32 or \
            row_limit.numel() != 1 or row_limit.device.type != "cuda":
        raise TypeError("row_limit must be a one-element int32 GPU tensor")
    return row_limit.data_ptr()


def combine(y, route_rows, topk_w, route_mask, out=None, row_limit=None):
    """moe_combine: out[t] = sum over read j of w[t,j] * y[route_rows[t*k+j]] (fp32).

    Route r is read when its mask is set and, with row_limit (offsets[E:E+1]
    of the route table), its row lies below offsets[E]."""
    torch = _torch()
    lib = _lib.load()
    _need(y, "y", torch.float32, 2)
    _need(route_rows, "route_rows", torch.int32, 1)
    _need(topk_w, "topk_w", torch.float32, 2)
    if route_mask is not None:
        _need(route_mask, "route_mask", torch.uint8, 2)
    lim = _row_limit(row_limit)
    T, k = topk_w.shape
    d = y.shape[1]
    if out is None:
        out = torch.empty(T, d, dtype=torch.float32, device=y.device)
    _need(out, "out", torch.float32, 2)
    rc = lib.moe_combine(_ptr(y), _ptr(route_rows), _ptr(topk_w), _ptr(route_mask), lim, T, k,
                         d, _ptr(out), _stream())
    _lib.check(rc, "moe_combine")
    return out


def combine_shared(y, route_rows, topk_w, route_mask, shared=None, out=None, out_bf16=None,
                   want_fp32=True, want_bf16=False, row_limit=None):
    """moe_combine_shared: routed combine plus the shared-expert rows, as fp32
    and/or bf16 (round to nearest even)."""
    torch = _torch()
    lib = _lib.load()
    _need(y, "y", torch.float32, 2)
    _need(route_rows, "route_rows", torch.int32, 1)
    _need(topk_w, "topk_w", torch.float32, 2)
    if route_mask is not None:
        _need(route_mask, "route_mask", torch.uint8, 2)
    lim = _row_limit(row_limit)
    T, k = topk_w.shape
    d = y.shape[1]
    if shared is not None:
        _need(shared, "shared", torch.float32, 2)
        if tuple(shared.shape) != (T, d):
            raise ValueError("shared must be [T, d]")
    if out is None and want_fp32:
        out = torch.empty(T, d, dtype=torch.float32, device=y.device)
    if out_bf16 is None and want_bf16:
        out_bf16 = torch.empty(T, d, dtype=torch.bfloat16, device=y.device)
    if out is not None:
        _need(out, "out", torch.float32, 2)
    if out_bf16 is not None:
        _need(out_bf16, "out_bf16", torch.bfloat16, 2)
    rc = lib.moe_combine_shared(_ptr(y), _ptr(route_rows), _ptr(topk_w), _ptr(route_mask), lim,
                                _ptr(shared), T, k, d, _ptr(out), _ptr(out_bf16), _stream())
    _lib.check(rc, "moe_combine_shared")
    return out, out_bf16


def quant_rows_fp8(x, q=None, s=None):
    """moe_quant_rows_fp8: per-row E4M3 codes and fp32 scales of a bf16 matrix."""
    torch = _torch()
    lib = _lib.load()
    _need(x, "x", torch.bfloat16, 2)
    rows, cols = x.shape
    if q is None:
        q = torch.empty(rows, cols, dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty(rows, dtype=torch.float32, device=x.device)
    rc = lib.moe_quant_rows_fp8(_ptr(x), rows, cols, _ptr(q), _ptr(s), _stream())
    _lib.check(rc, "moe_quant_rows_fp8")
    return q, s


def _need_rows(t, name, shape, dtypes, device):
    """A contiguous tensor of the given shape, of one of the given types and
    on the given device."""
    try:
        if t.dtype in dtypes and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _on_current(t, name):
    """The device of t, which has to be the current one: the kernels run on
    its current stream."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be on a GPU device")
    if dev.index != torch._C._cuda_getDevice():  # torch.cuda.current_device(), initialised by x
        raise ValueError(f"{name} is on {dev}, which is not the current device")
    return dev


def add_rmsnorm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, y=None, q=None,
                s=None, want_bf16=True, want_fp8=False):
    """moe_add_rmsnorm: v = residual + x, and the root-mean-square norm of v.

    x [rows, d] and residual (optional) are bf16 or fp32, weight [d] likewise.
    Returns (y, residual_out, q, s): the norm in bf16, the sum v in the
    residual's type, E4M3 codes (uint8) and row scales of the norm -- None for
    what is not wanted.  residual_out may be residual itself; without a
    residual it is written only if given (then v is x).  No rows: nothing is
    launched."""
    torch = _torch()
    native = _native()
    if native is not None and getattr(x, "is_cuda", False):
        dev = torch._C._cuda_getDevice()
        done = native.add_rmsnorm(x, weight, eps, residual, residual_out, y, q, s, want_bf16,
                                  want_fp8, dev, torch._C._cuda_getCurrentRawStream(dev))
        if type(done) is tuple:
            return done
        if done is not None:  # the launch's status: the kernel may have run, once is all
            _lib.check(done, "moe_add_rmsnorm")
    # refusals, no rows, and without the module every call
    lib = _lib.load()
    dev = _on_current(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dims, got {x.dim()}")
    shape, kinds = x.shape, (torch.bfloat16, torch.float32)
    rows, d = shape
    _need_rows(x, "x", shape, kinds, dev)
    _need_rows(weight, "weight", shape[1:], kinds, dev)
    if residual is not None:
        _need_rows(residual, "residual", shape, kinds, dev)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
    if residual_out is not None:
        _need_rows(residual_out, "residual_out", shape,
                   ((x if residual is None else residual).dtype,), dev)
    if y is None:
        if want_bf16:
            y = torch.empty_like(x, dtype=torch.bfloat16)
    else:
        _need_rows(y, "y", shape, (torch.bfloat16,), dev)
    if q is not None:
        _need_rows(q, "q", shape, (torch.uint8,), dev)
    elif want_fp8 or s is not None:
        q = torch.empty_like(x, dtype=torch.uint8)
    if s is not None:
        _need_rows(s, "s", shape[:1], (torch.float32,), dev)
    elif q is not None:
        s = torch.empty(rows, dtype=torch.float32, device=dev)
    if rows == 0:
        return y, residual_out, q, s
    f32 = torch.float32
    rdt = (x if residual is None else residual).dtype
    rc = lib.moe_add_rmsnorm(x.data_ptr(), int(x.dtype == f32), _ptr(residual),
                             _ptr(residual_out), int(rdt == f32), weight.data_ptr(),
                             int(weight.dtype == f32), eps, rows, d, _ptr(y), _ptr(q), _ptr(s),
                             _stream())
    _lib.check(rc, "moe_add_rmsnorm")
    return y, residual_out, q, s


def decode_ffn(x, topk_ids, topk_w, route_mask, w_gate, w_up, w_down, s_gate, s_up, s_down,
               shared=None, out=None, out_dtype=None, workspace=None):
    """moe_decode_ffn: the routed experts of a few tokens (T * k at most
    MOE_DECODE_MAX_ROUTES) with MXFP4 weights, straight from the ids.

    out [T, d] is fp32 or bf16; if it is not given, it is made in out_dtype
    (torch.float32 by default).  The other arguments are those of route_build,
    grouped_ffn and combine_shared."""
    torch = _torch()
    native = _native()
    if (native is not None and out is not None and workspace is not None
            and getattr(x, "is_cuda", False)):
        dev = torch._C._cuda_getDevice()
        done = native.decode_ffn(x, topk_ids, topk_w, route_mask, w_gate, w_up, w_down, s_gate,
                                 s_up, s_down, shared, out, workspace, dev,
                                 torch._C._cuda_getCurrentRawStream(dev))
        if done is True:
            return out
        if done is not None:  # the launch's status, as in add_rmsnorm
            _lib.check(done, "moe_decode_ffn")
    # outputs to be made, refusals, and without the module every call
    lib = _lib.load()
    dev = _on_current(x, "x")
    if x.dim() != 2 or not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 3:
        raise ValueError("x must have 2 dims and w_gate 3")
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids must have 2 dims")
    T, d = x.shape
    E, f, _ = w_gate.shape
    k = topk_ids.shape[1]
    if T == 0:
        raise ValueError("x must have at least one row")
    _need_rows(x, "x", (T, d), (torch.bfloat16,), dev)
    _need_rows(topk_ids, "topk_ids", (T, k), (torch.int32,), dev)
    _need_rows(topk_w, "topk_w", (T, k), (torch.float32,), dev)
    if route_mask is not None:
        _need_rows(route_mask, "route_mask", (T, k), (torch.uint8,), dev)
    for name, t, shape in (("w_gate", w_gate, (E, f, d // 2)), ("w_up", w_up, (E, f, d // 2)),
                           ("w_down", w_down, (E, d, f // 2)), ("s_gate", s_gate, (E, f, d // 32)),
                           ("s_up", s_up, (E, f, d // 32)), ("s_down", s_down, (E, d, f // 32))):
        _need_rows(t, name, shape, (torch.uint8,), dev)
    if shared is not None:
        _need_rows(shared, "shared", (T, d), (torch.float32,), dev)
    if out is None:
        out = torch.empty(T, d, dtype=out_dtype or torch.float32, device=dev)
    _need_rows(out, "out", (T, d), (torch.float32, torch.bfloat16), dev)
    desc = ctypes.byref(ffn_desc(T, k, E, d, f, weights="mxfp4"))
    if workspace is None:
        workspace = torch.empty(max(lib.moe_decode_ffn_workspace(desc), 256), dtype=torch.uint8,
                                device=dev)
    _need_rows(workspace, "workspace", workspace.shape, (torch.uint8,), dev)
    f32 = out.dtype == torch.float32
    rc = lib.moe_decode_ffn(desc, x.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(),
                            _ptr(route_mask), w_gate.data_ptr(), w_up.data_ptr(),
                            w_down.data_ptr(), s_gate.data_ptr(), s_up.data_ptr(),
                            s_down.data_ptr(), _ptr(shared), out.data_ptr() if f32 else None,
                            None if f32 else out.data_ptr(), workspace.data_ptr(),
                            workspace.numel(), _stream())
    _lib.check(rc, "moe_decode_ffn")
    return out


# scores of route_select by name
_SCORES = {"softmax": MOE_SCORES_SOFTMAX, "sigmoid": MOE_SCORES_SIGMOID}


def _int32(value, name) -> int:
    """value as the C ABI's ints hold it (ctypes would drop the bits above)."""
    value = operator.index(value)
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def route_select(logits, k: int, scores: str = "sigmoid", bias=None, groups: int = 1,
                 top_groups: int = 1, group_top: int = 2, renormalise: bool = True,
                 scale: float = 1.0, topk_ids=None, topk_w=None):
    """moe_route_select: the k experts of largest score + bias, out of the
    top_groups best of `groups` groups, and the gates of their scores.

    logits [T, E] are fp32 or bf16 (-inf: out of service), scores "sigmoid" or
    "softmax" over all E, bias fp32 [E] chooses only.  A group's value is the sum
    of its group_top (1 or 2) largest choices.  Returns (topk_ids, topk_w), what
    route_build, combine and MoEPrefill take.  No rows: nothing is launched."""
    torch = _torch()
    native = _native()
    if native is not None and getattr(logits, "is_cuda", False):
        dev = torch._C._cuda_getDevice()
        done = native.route_select(logits, k, _SCORES.get(scores), bias, groups, top_groups,
                                   group_top, bool(renormalise), scale, topk_ids, topk_w, dev,
                                   torch._C._cuda_getCurrentRawStream(dev))
        if type(done) is tuple:
            return done
        if done is not None:  # the launch's status, as in add_rmsnorm
            _lib.check(done, "moe_route_select")
    lib = _lib.load()
    dev = _on_current(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must have 2 dims, got {logits.dim()}")
    if scores not in _SCORES:
        raise ValueError(f"scores must be one of {sorted(_SCORES)}, got {scores!r}")
    f32 = torch.float32
    _need_rows(logits, "logits", logits.shape, (f32, torch.bfloat16), dev)
    T, E = logits.shape
    k, groups, top_groups, group_top = (
        _int32(v, n) for v, n in ((k, "k"), (groups, "groups"), (top_groups, "top_groups"),
                                  (group_top, "group_top")))
    if k < 1:
        raise ValueError(f"k must be at least 1, got {k}")
    if bias is not None:
        _need_rows(bias, "bias", (E,), (f32,), dev)
    if topk_ids is None:
        topk_ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty(T, k, dtype=f32, device=dev)
    _need_rows(topk_ids, "topk_ids", (T, k), (torch.int32,), dev)
    _need_rows(topk_w, "topk_w", (T, k), (f32,), dev)
    if T == 0:
        return topk_ids, topk_w
    desc = _lib.MoeSelectDesc(T, _int32(E, "E"), k, int(logits.dtype == f32), _SCORES[scores],
                              groups, top_groups, group_top, bool(renormalise), scale)
    rc = lib.moe_route_select(ctypes.byref(desc), logits.data_ptr(), _ptr(bias),
                              topk_ids.data_ptr(), topk_w.data_ptr(), _stream())
    _lib.check(rc, "moe_route_select")
    return topk_ids, topk_w


def quant_blocks_fp8(x, q=None, s=None):
    """moe_quant_blocks_fp8: E4M3 codes (uint8) of bf16 or fp32 rows [rows, cols]
    and fp32 scales [rows, cols / 128], one for each block of 128 columns.  No
    rows: nothing is launched."""
    torch = _torch()
    native = _native()
    if native is not None and getattr(x, "is_cuda", False):
        dev = torch._C._cuda_getDevice()
        done = native.quant_blocks_fp8(x, q, s, dev, torch._C._cuda_getCurrentRawStream(dev))
        if type(done) is tuple:
            return done
        if done is not None:  # the launch's status, as in add_rmsnorm
            _lib.check(done, "moe_quant_blocks_fp8")
    lib = _lib.load()
    dev = _on_current(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dims, got {x.dim()}")
    rows, cols = x.shape
    _need_rows(x, "x", x.shape, (torch.bfloat16, torch.float32), dev)
    if cols % 128 != 0:
        raise ValueError(f"x must have a multiple of 128 columns, got {cols}")
    if q is None:
        q = torch.empty(rows, cols, dtype=torch.uint8, device=dev)
    if s is None:
        s = torch.empty(rows, cols // 128, dtype=torch.float32, device=dev)
    _need_rows(q, "q", (rows, cols), (torch.uint8,), dev)
    _need_rows(s, "s", (rows, cols // 128), (torch.float32,), dev)
    if rows == 0:
        return q, s
    rc = lib.moe_quant_blocks_fp8(x.data_ptr(), int(x.dtype == torch.float32),
                                  _int32(rows, "rows"), _int32(cols, "cols"), q.data_ptr(),
                                  s.data_ptr(), _stream())
    _lib.check(rc, "moe_quant_blocks_fp8")
    return q, s


def _need_codes(x):
    """x as (rows, scales or None), checked: bf16 rows, or a pair of E4M3 codes
    and the scales of their blocks."""
    torch = _torch()
    xs = None
    if isinstance(x, tuple):
        if len(x) != 2:
            raise ValueError("x must be bf16 rows or a pair of codes and scales")
        x, xs = x
    dev = _on_current(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dims, got {x.dim()}")
    _need_rows(x, "x", x.shape, (torch.bfloat16 if xs is None else torch.uint8,), dev)
    if x.shape[1] % 128 != 0:
        raise ValueError(f"x must have a multiple of 128 columns, got {x.shape[1]}")
    if xs is not None:
        _need_rows(xs, "the scales of x", (x.shape[0], x.shape[1] // 128), (torch.float32,), dev)
    return x, xs


def _need_blocks(w, s, name, N, K, dev):
    """E4M3 codes [N, K] and a scale for each block of 128 x 128."""
    _need_rows(w, "w" + name, (N, K), (_torch().uint8,), dev)
    _need_rows(s, "s" + name, (-(-N // 128), K // 128), (_torch().float32,), dev)


def _need_out(out, out_dtype, shape, dev):
    torch = _torch()
    kinds = (torch.float32, torch.bfloat16)
    if out is None:
        if out_dtype not in (None, *kinds):
            raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16, got {out_dtype}")
        out = torch.empty(shape, dtype=out_dtype or torch.float32, device=dev)
    _need_rows(out, "out", shape, kinds, dev)
    return out


def _result_type(out, short) -> int:
    """out's type with the flag for short sums, as the C ABI takes them."""
    f32 = out.dtype == _torch().float32
    if short and f32:
        raise ValueError("short_sums is for bf16 results")
    return int(f32) | (MOE_SHORT_SUMS if short else 0)


def _need_ws(workspace, need, dev):
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _need_rows(workspace, "workspace", workspace.shape, (torch.uint8,), dev)
    return workspace


def matmul_fp8(x, w, s, out=None, out_dtype=None, workspace=None, short_sums: bool = False):
    """moe_matmul_fp8: x [M, K] times the transpose of 8-bit weights w [N, K].

    x: bf16 rows, quantised by the call, or the pair (codes, scales) of
    quant_blocks_fp8.  w: E4M3 codes (uint8), s: fp32 [ceil(N / 128), K / 128], a
    scale for each block of 128 x 128.  out [M, N] is fp32 or bf16; if it is not
    given, it is made in out_dtype (torch.float32 by default).  workspace is used
    for bf16 rows only.  No rows: nothing is launched.

    Sums are fp32's.  short_sums, for bf16 results: they may keep of eight products
    what lies within 13 bits of the largest, which is twice as fast for many rows."""
    torch = _torch()
    native = _native()
    rows, xs = x if type(x) is tuple and len(x) == 2 else (x, None)
    short = bool(short_sums)  # such calls are not worth the module's short way
    if native is not None and getattr(rows, "is_cuda", False):
        dev = torch._C._cuda_getDevice()
        done = native.matmul_fp8(rows, xs, w, s, out, out_dtype in (None, torch.float32),
                                 short or (out is None and out_dtype not in (None, torch.float32, torch.bfloat16)),
                                 workspace, dev, torch._C._cuda_getCurrentRawStream(dev))
        if type(done) is int:  # the launch's status, as in add_rmsnorm
            _lib.check(done, "moe_matmul_fp8")
        if done is not None:
            return done
    lib = _lib.load()
    x, xs = _need_codes(x)
    dev = x.device
    M, K = (_int32(v, "a size of x") for v in x.shape)
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a tensor of 2 dims")
    N = _int32(w.shape[0], "N")
    _need_blocks(w, s, "", N, K, dev)
    out = _need_out(out, out_dtype, (M, N), dev)
    kind = _result_type(out, short)
    if M == 0:
        return out
    if xs is None:
        workspace = _need_ws(workspace, lib.moe_matmul_fp8_workspace(M, N, K), dev)
    else:
        workspace = None
    rc = lib.moe_matmul_fp8(x.data_ptr(), _ptr(xs), M, N, K, w.data_ptr(), s.data_ptr(),
                            out.data_ptr(), kind, _ptr(workspace),
                            0 if workspace is None else workspace.numel(), _stream())
    _lib.check(rc, "moe_matmul_fp8")
    return out


def shared_ffn(x, w_gate, w_up, w_down, s_gate, s_up, s_down, out=None, out_dtype=None,
               workspace=None, short_sums: bool = False):
    """moe_shared_ffn: the shared expert, Wd . (silu(Wg . x) * (Wu . x)), whose rows
    are the `shared` of combine_shared, decode_ffn and MoEPrefill.

    x [T, d], out [T, d] and short_sums (of the down product) as for matmul_fp8;
    w_gate, w_up [f, d] and w_down [d, f] E4M3 codes (uint8), their scales fp32 for
    each block of 128 x 128."""
    torch = _torch()
    native = _native()
    rows, xs = x if type(x) is tuple and len(x) == 2 else (x, None)
    short = bool(short_sums)  # such calls are not worth the module's short way
    if native is not None and getattr(rows, "is_cuda", False):
        dev = torch._C._cuda_getDevice()
        done = native.shared_ffn(rows, xs, w_gate, w_up, w_down, s_gate, s_up, s_down, out,
                                 out_dtype in (None, torch.float32),
                                 short or (out is None and out_dtype not in (None, torch.float32, torch.bfloat16)),
                                 workspace, dev, torch._C._cuda_getCurrentRawStream(dev))
        if type(done) is int:  # the launch's status, as in add_rmsnorm
            _lib.check(done, "moe_shared_ffn")
        if done is not None:
            return done
    lib = _lib.load()
    x, xs = _need_codes(x)
    dev = x.device
    T, d = (_int32(v, "a size of x") for v in x.shape)
    if not isinstance(w_gate, torch.Tensor) or w_gate.dim() != 2:
        raise ValueError("w_gate must be a tensor of 2 dims")
    f = _int32(w_gate.shape[0], "f")
    if f % 128 != 0:
        raise ValueError(f"w_gate must have a multiple of 128 rows, got {f}")
    _need_blocks(w_gate, s_gate, "_gate", f, d, dev)
    _need_blocks(w_up, s_up, "_up", f, d, dev)
    _need_blocks(w_down, s_down, "_down", d, f, dev)
    out = _need_out(out, out_dtype, (T, d), dev)
    kind = _result_type(out, short)
    if T == 0:
        return out
    workspace = _need_ws(workspace, lib.moe_shared_ffn_workspace(T, d, f), dev)
    rc = lib.moe_shared_ffn(x.data_ptr(), _ptr(xs), T, d, f, w_gate.data_ptr(), w_up.data_ptr(),
                            w_down.data_ptr(), s_gate.data_ptr(), s_up.data_ptr(),
                            s_down.data_ptr(), out.data_ptr(), kind, workspace.data_ptr(),
                            workspace.numel(), _stream())
    _lib.check(rc, "moe_shared_ffn")
    return out


class MoEPrefill:
    """The whole path -- route build, grouped FFN, combine -- with buffers kept
    across calls (nothing is allocated per call after construction).

    weights: "bf16", "fp8" or "mxfp4" (default: by fp8).  out_dtype:
    torch.float32 (default) or torch.bfloat16.  With MXFP4 weights and few
    routes (_decodes) a pass is decode_ffn, unless stage events are asked
    for or self.decode is set to False: self.rt and self.y are then not written.
    decode_ffn keeps 16 bits of h, the grouped path 8: a token's output differs
    by up to about 2^-8 of its norm between the two, on top of the order of sums.
    A program that needs one answer for both sets decode to False."""

    DECODE_ROUTES = 64  # the most that decode_ffn takes

    @classmethod
    def _decodes(cls, T: int, k: int, E: int, d: int, f: int) -> bool:
        """Whether decode_ffn is the faster way, as far as shapes tell.

        It reads an expert's weights again for every four rows (gate/up) and
        every two (down); the grouped path reads them once and has three
        launches more.  MI355X, us (grouped in brackets); zipf: routers with
        favourites; same: every token to the same k experts.

        At d 4096, f 2048 up to 24 tokens and 32 routes it is the faster one
        whatever the ids: 24 routes over 256 experts 62 (77), same 26 (49);
        32 over 8 41 (47), zipf 46 (48), same 43 (50); 24 of one expert 59 (62).
        32 tokens of one route each gain while they have experts to go to: over
        8 40 (47), zipf 44 (48), all to one 77 (62); over 4 47 (49), zipf 46
        (49); over 2 44 (50), zipf 68 (62).  More routes pay while there are
        experts for them: 60 over 256 144 (169), zipf 123 (164), same 57 (50);
        40 over 32 81 (82); 40 over 16 56 (53); 64 over 16 73 (53), over 8 72
        (48).  With more tokens too much hangs on the ids: 64 tokens over 256
        experts 148 (172), all to one 150 (65).  Narrow layers are launches
        mostly: d 1024, f 512, 64 routes over 16 experts 21 (28), zipf 26 (29),
        same 33 (33)."""
        R = T * k
        if R > cls.DECODE_ROUTES or T > 32:
            return False
        return d * f <= 1 << 19 or 2 * R <= 3 * E or (R <= 32 and (T <= 24 or E >= 4))

    def __init__(self, T: int, k: int, E: int, d: int, f: int, fp8: bool = False, device="cuda",
                 weights: Optional[str] = None, out_dtype=None):
        torch = _torch()
        lib = _lib.load()
        if out_dtype not in (None, torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16, got {out_dtype}")
        self.T, self.k, self.E, self.d, self.f = T, k, E, d, f
        self.weights = weights or ("fp8" if fp8 else "bf16")
        self.fp8 = self.weights == "fp8"
        dev = torch.device(device)
        R = T * k
        self.rt = RouteTable(
            counts=torch.empty(E + 1, dtype=torch.int32, device=dev),
            offsets=torch.empty(E + 2, dtype=torch.int32, device=dev),
            sorted_routes=torch.empty(R, dtype=torch.int32, device=dev),
            route_rows=torch.empty(R, dtype=torch.int32, device=dev),
        )
        self.rb_ws = torch.empty(max(lib.moe_route_build_workspace(T, k, E), 256),
                                 dtype=torch.uint8, device=dev)
        self.desc = ffn_desc(T, k, E, d, f, fp8, weights)
        self.ffn_ws = _ffn_ws(self.desc, dev, None)
        more = lib.moe_decode_ffn_workspace(ctypes.byref(self.desc))  # 0: not its kind of layer
        if more > self.ffn_ws.numel():
            self.ffn_ws = torch.empty(more, dtype=torch.uint8, device=dev)
        self.y = torch.empty(R, d, dtype=torch.float32, device=dev)
        self.out = torch.empty(T, d, dtype=out_dtype or torch.float32, device=dev)
        # offsets[E]: rows of y the FFN writes.  The combine reads no route at
        # or past it, so active routes whose ids lie outside [0, E) -- which
        # the route build sends to the trailing bin -- add exact zeros, as
        # masked ones do.
        self.row_limit = self.rt.offsets[E:E + 1]
        self.decode = self.weights == "mxfp4" and self._decodes(T, k, E, d, f)

    def __call__(self, x, topk_ids, topk_w, route_mask, w_gate, w_up, w_down, s_gate=None,
                 s_up=None, s_down=None, stage_events=None, shared=None):
        """One pass of the path.  x: bf16 rows [T, d], or with fp8 weights the
        pair of their E4M3 codes and scales (add_rmsnorm, quant_rows_fp8).
        shared: fp32 rows [T, d] of the shared expert, added to the routed
        sum.  stage_events: optional torch events recorded on the current
        stream: 2 events around the gate/up stage, or 6 -- before the route
        build and after each of route build, FFN plan, gate/up, down and
        combine."""
        ev = stage_events
        if isinstance(x, tuple):
            if not self.fp8 or ev is not None:
                raise ValueError("codes and scales need fp8 weights, and no stage events")
            rt = route_build(topk_ids, route_mask, self.E, out=self.rt, workspace=self.rb_ws)
            grouped_ffn_codes(*x, rt.offsets, rt.sorted_routes, w_gate, w_up, w_down, self.k,
                              s_gate, s_up, s_down, y=self.y, workspace=self.ffn_ws)
            return self._combine(rt, topk_w, route_mask, shared)
        if self.decode and ev is None:
            return decode_ffn(x, topk_ids, topk_w, route_mask, w_gate, w_up, w_down, s_gate, s_up,
                              s_down, shared=shared, out=self.out, workspace=self.ffn_ws)
        if ev is not None and len(ev) == 2:
            ev = [None, None, ev[0], ev[1], None, None]  # around ffn_gate_up
        if ev is not None and ev[0] is not None:
            ev[0].record()
        rt = route_build(topk_ids, route_mask, self.E, out=self.rt, workspace=self.rb_ws)
        if ev is None:
            grouped_ffn(x, rt.offsets, rt.sorted_routes, w_gate, w_up, w_down, self.k, s_gate,
                        s_up, s_down, y=self.y, workspace=self.ffn_ws)
            return self._combine(rt, topk_w, route_mask, shared)

        def mark(i):
            if ev[i] is not None:
                ev[i].record()

        mark(1)
        ffn_plan(self.desc, x, rt.offsets, self.ffn_ws)
        mark(2)
        ffn_gate_up(self.desc, x, rt.sorted_routes, w_gate, w_up, s_gate, s_up, self.ffn_ws)
        mark(3)
        ffn_down(self.desc, rt.offsets, w_down, s_down, self.y, self.ffn_ws)
        mark(4)
        out = self._combine(rt, topk_w, route_mask, shared)
        mark(5)
        return out

    def _combine(self, rt, topk_w, route_mask, shared):
        torch = _torch()
        if shared is None and self.out.dtype == torch.float32:
            return combine(self.y, rt.route_rows, topk_w, route_mask, out=self.out,
                           row_limit=self.row_limit)
        f32 = self.out.dtype == torch.float32
        combine_shared(self.y, rt.route_rows, topk_w, route_mask, shared=shared,
                       out=self.out if f32 else None, out_bf16=None if f32 else self.out,
                       want_fp32=f32, row_limit=self.row_limit)
        return self.out

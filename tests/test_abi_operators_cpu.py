"""The C ABI of the norm and of the 4-bit expert calls on the host: bad
arguments are rejected with the documented status before the GPU is touched
(no call here passes validation)."""
import ctypes
import os

import pytest

from routed_expert_prefill_amd import _lib

A = 0x10000000  # a 16-byte-aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return _lib.load()


def test_add_rmsnorm_errors(lib):
    def f(x=A, xt=0, r=0, ro=0, rt=0, w=A, wt=0, eps=1e-6, rows=4, d=256, y=A, q=0, s=0):
        return lib.moe_add_rmsnorm(x or None, xt, r or None, ro or None, rt, w or None, wt, eps,
                                   rows, d, y or None, q or None, s or None, None)

    assert f(x=0) == _lib.MOE_EINVAL
    assert f(w=0) == _lib.MOE_EINVAL
    assert f(y=0) == _lib.MOE_EINVAL  # no output
    assert f(q=A) == _lib.MOE_EINVAL  # codes without scales
    assert f(s=A) == _lib.MOE_EINVAL  # scales without codes
    assert f(rows=0) == _lib.MOE_EINVAL
    assert f(d=0) == _lib.MOE_EINVAL
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert f(eps=eps) == _lib.MOE_EINVAL
    assert f(xt=2) == _lib.MOE_EUNSUPPORTED
    assert f(wt=-1) == _lib.MOE_EUNSUPPORTED
    assert f(rt=3) == _lib.MOE_EUNSUPPORTED
    assert f(ro=A, rt=1) == _lib.MOE_EUNSUPPORTED  # no residual: residual_out has x's type
    assert f(d=252) == _lib.MOE_EUNSUPPORTED
    assert f(d=16392) == _lib.MOE_EUNSUPPORTED
    for name in ("x", "r", "ro", "w", "y"):
        assert f(**{name: A + 8}) == _lib.MOE_EALIGN
    assert f(q=A + 8, s=A) == _lib.MOE_EALIGN
    assert f(q=A, s=A + 4) == _lib.MOE_EALIGN


def _desc(T=32, k=6, E=16, d=512, f=256, w=_lib.MOE_W_MXFP4, a=_lib.MOE_ACT_BF16):
    return _lib.MoeFfnDesc(T, k, E, d, f, w, a)


def test_mxfp4_ffn_errors(lib):
    def f(desc=None, x=A, wg=A, sg=A, su=A, sd=A, ws=A, wsb=1 << 40):
        return lib.moe_grouped_ffn(ctypes.byref(desc or _desc()), x, A, A, wg, A, A, sg or None,
                                   su or None, sd or None, A, ws or None, wsb, None)

    q = lambda **kw: lib.moe_grouped_ffn_workspace(ctypes.byref(_desc(**kw)))  # noqa: E731
    assert q() >= q(w=_lib.MOE_W_BF16) > 0  # h and the tile list, as with bf16 weights
    assert q(a=_lib.MOE_ACT_FP8_E4M3_ROW) == 0 and q(w=3) == 0
    for s in ("sg", "su", "sd"):
        assert f(**{s: 0}) == _lib.MOE_EINVAL  # scales are needed
        assert f(**{s: A + 8}) == _lib.MOE_EALIGN
    assert f(desc=_desc(a=_lib.MOE_ACT_FP8_E4M3_ROW)) == _lib.MOE_EUNSUPPORTED
    assert f(desc=_desc(d=192)) == _lib.MOE_EUNSUPPORTED
    assert f(wg=A + 8) == _lib.MOE_EALIGN
    assert f(ws=0) == _lib.MOE_EWORKSPACE and f(wsb=4096) == _lib.MOE_EWORKSPACE
    d = ctypes.byref(_desc())
    assert lib.moe_ffn_gate_up(d, A, A, A, A, None, A, A, 1 << 40, None) == _lib.MOE_EINVAL
    assert lib.moe_ffn_down(d, A, A, None, A, A, 1 << 40, None) == _lib.MOE_EINVAL


def test_decode_errors(lib):
    def f(desc=None, ws=A, wsb=1 << 30, **kw):
        names = ("x", "ids", "w", "mask", "wg", "wu", "wd", "sg", "su", "sd", "shared", "out",
                 "out_bf16")
        p = {**dict.fromkeys(names, A), "mask": 0, "shared": 0, "out_bf16": 0, **kw}
        return lib.moe_decode_ffn(ctypes.byref(desc or _desc(T=2)), *[p[n] or None for n in names],
                                  ws or None, wsb, None)

    q = lambda **kw: lib.moe_decode_ffn_workspace(ctypes.byref(_desc(**kw)))  # noqa: E731
    assert q(T=1) >= 6 * 256 * 2
    assert q(T=16, k=4) > 0 and q(T=13, k=5) == 0  # 64 routes, 65
    assert q(T=2, w=0) == 0 and q(T=2, w=1, a=1) == 0 and q(T=0) == 0
    for n in ("x", "ids", "w", "wg", "wu", "wd", "sg", "su", "sd", "out"):
        assert f(**{n: 0}) == _lib.MOE_EINVAL, n
        assert f(**{n: A + 8}) == _lib.MOE_EALIGN, n
    for n in ("mask", "shared", "out_bf16"):
        assert f(**{n: A + 8}) == _lib.MOE_EALIGN, n
    assert f(desc=_desc(T=11)) == _lib.MOE_EUNSUPPORTED  # 66 routes
    assert f(desc=_desc(T=2, w=_lib.MOE_W_BF16)) == _lib.MOE_EUNSUPPORTED
    assert f(desc=_desc(T=2, d=320)) == _lib.MOE_EUNSUPPORTED
    assert f(desc=_desc(T=0)) == _lib.MOE_EINVAL
    assert f(ws=0) == _lib.MOE_EWORKSPACE and f(wsb=1024) == _lib.MOE_EWORKSPACE
    assert lib.moe_decode_ffn(None, *[A] * 14, 1 << 30, None) == _lib.MOE_EINVAL


def test_grouped_ffn_codes_errors(lib):
    names = ("xq", "xs", "offs", "sr", "wg", "wu", "wd", "sg", "su", "sd", "y")

    def f(desc=None, ws=A, wsb=1 << 40, **kw):
        p = {**dict.fromkeys(names, A), **kw}
        d = desc or _desc(w=_lib.MOE_W_FP8_E4M3_B128, a=_lib.MOE_ACT_FP8_E4M3_ROW)
        return lib.moe_grouped_ffn_codes(ctypes.byref(d), *[p[n] or None for n in names],
                                         ws or None, wsb, None)

    for n in names:
        assert f(**{n: 0}) == _lib.MOE_EINVAL, n
        assert f(**{n: A + 8}) == _lib.MOE_EALIGN, n
    assert f(desc=_desc()) == _lib.MOE_EUNSUPPORTED  # MXFP4
    assert f(desc=_desc(w=0, a=0)) == _lib.MOE_EUNSUPPORTED
    assert f(desc=_desc(T=0, w=1, a=1)) == _lib.MOE_EINVAL
    assert f(ws=0) == _lib.MOE_EWORKSPACE and f(wsb=4096) == _lib.MOE_EWORKSPACE
    assert f(ws=A + 8) == _lib.MOE_EALIGN

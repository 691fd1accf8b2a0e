"""The C ABI of expert selection, block quantisation, 8-bit products and the
shared expert on the host: bad arguments are rejected with the documented status
before the GPU is touched (no call here passes validation)."""
import ctypes
import os

import pytest

from routed_expert_prefill_amd import _lib

A = 0x10000000  # a 16-byte-aligned fake device address (never dereferenced)
INVAL, UNSUP, ALIGN, WS = (_lib.MOE_EINVAL, _lib.MOE_EUNSUPPORTED, _lib.MOE_EALIGN,
                           _lib.MOE_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return _lib.load()


def test_route_select_errors(lib):
    def f(z=A, b=0, ids=A, w=A, **kw):
        d = dict(T=4, E=16, k=2, logits_dtype=1, scores=1, groups=4, top_groups=2, group_top=2,
                 renormalise=1, scale=1.0)
        d.update(kw)
        return lib.moe_route_select(ctypes.byref(_lib.MoeSelectDesc(**d)), z or None, b or None,
                                    ids or None, w or None, None)

    assert lib.moe_route_select(None, A, None, A, A, None) == INVAL
    for n in ("z", "ids", "w"):
        assert f(**{n: 0}) == INVAL and f(**{n: A + 8}) == ALIGN, n
    assert f(b=A + 4) == ALIGN
    for n in ("T", "E", "k", "groups", "top_groups"):
        assert f(**{n: 0}) == INVAL and f(**{n: -1}) == INVAL, n
    assert f(T=1 << 27) == INVAL
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert f(scale=scale) == INVAL
    for bad in (dict(logits_dtype=2), dict(logits_dtype=-1), dict(scores=2), dict(scores=-1),
                dict(E=260), dict(k=17, E=64, top_groups=4), dict(k=9), dict(groups=3),
                dict(top_groups=5), dict(group_top=0), dict(group_top=3),
                dict(E=130, groups=65, top_groups=65)):
        assert f(**bad) == UNSUP, bad


def test_quant_blocks_errors(lib):
    def f(x=A, t=0, rows=4, cols=256, q=A, s=A):
        return lib.moe_quant_blocks_fp8(x or None, t, rows, cols, q or None, s or None, None)

    for n in ("x", "q", "s"):
        assert f(**{n: 0}) == INVAL and f(**{n: A + 8}) == ALIGN, n
    assert f(rows=0) == INVAL and f(cols=0) == INVAL
    assert f(cols=192) == UNSUP and f(t=2) == UNSUP and f(t=-1) == UNSUP


def test_matmul_errors(lib):
    def f(x=A, xs=0, M=4, N=100, K=256, w=A, ws=A, y=A, t=1, room=A, bytes=1 << 30):
        return lib.moe_matmul_fp8(x or None, xs or None, M, N, K, w or None, ws or None, y or None,
                                  t, room or None, bytes, None)

    q = lib.moe_matmul_fp8_workspace
    assert q(0, 1, 128) == 0 and q(1, 0, 128) == 0 and q(1, 1, 64) == 0
    assert q(1, 1, (1 << 20) + 128) == 0
    assert q(5, 7, 256) >= 5 * 256 + 5 * 2 * 4 and q(5, 7, 256) % 256 == 0
    assert q(1 << 20, 1, 1 << 20) > 1 << 40  # beyond 32 bits
    for n in ("x", "w", "ws", "y"):
        assert f(**{n: 0}) == INVAL and f(**{n: A + 8}) == ALIGN, n
    assert f(xs=A + 4) == ALIGN and f(room=A + 8) == ALIGN
    for n in ("M", "N", "K"):
        assert f(**{n: 0}) == INVAL and f(**{n: -5}) == INVAL, n
    assert f(K=192) == UNSUP and f(K=1 << 21) == UNSUP and f(t=2) == UNSUP and f(t=-1) == UNSUP
    assert f(M=(1 << 31) - 1, N=1 << 20, K=128) == UNSUP
    assert f(room=0) == WS and f(bytes=4 * 256) == WS


def test_shared_errors(lib):
    names = ("x", "wg", "wu", "wd", "sg", "su", "sd", "out")

    def f(xs=0, T=4, d=256, f=128, t=1, room=A, bytes=1 << 30, **kw):
        p = {**dict.fromkeys(names, A), **kw}
        return lib.moe_shared_ffn(p["x"] or None, xs or None, T, d, f,
                                  *[p[n] or None for n in names[1:]], t, room or None, bytes, None)

    q = lib.moe_shared_ffn_workspace
    assert q(0, 128, 128) == 0 and q(1, 192, 128) == 0 and q(1, 128, 64) == 0
    assert 0 < q(1, 256, 128) < q(64, 256, 128)
    for n in names:
        assert f(**{n: 0}) == INVAL and f(**{n: A + 8}) == ALIGN, n
    assert f(xs=A + 8) == ALIGN and f(room=A + 8) == ALIGN
    assert f(T=0) == INVAL and f(d=0) == INVAL and f(f=-128) == INVAL
    assert f(d=320) == UNSUP and f(f=100) == UNSUP and f(t=3) == UNSUP and f(d=1 << 21) == UNSUP
    assert f(room=0) == WS and f(bytes=256) == WS

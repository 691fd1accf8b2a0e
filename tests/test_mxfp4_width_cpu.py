"""MXFP4 rows too wide for the kernels' 32-bit offsets are refused on the host."""
import ctypes

import pytest

from routed_expert_prefill_amd import _lib
from test_abi_operators_cpu import A, _desc, lib  # noqa: F401

MOST = 1 << 24


@pytest.mark.parametrize("d,f,ok", [(MOST, 128, True), (128, MOST, True), (MOST + 128, 128, False),
                                    (128, MOST + 128, False), (1 << 26, 128, False),
                                    (128, 1 << 30, False)])
def test_widest_rows(lib, d, f, ok):  # noqa: F811
    desc = ctypes.byref(_desc(T=1, k=1, d=d, f=f))
    assert (lib.moe_grouped_ffn_workspace(desc) > 0) == ok
    assert (lib.moe_decode_ffn_workspace(desc) > 0) == ok
    # no workspace: the last check of a call that is otherwise good
    want = _lib.MOE_EWORKSPACE if ok else _lib.MOE_EUNSUPPORTED
    assert lib.moe_grouped_ffn(desc, *[A] * 10, None, 0, None) == want
    assert lib.moe_ffn_plan(desc, A, A, None, 0, None) == want
    assert lib.moe_decode_ffn(desc, A, A, A, None, *[A] * 6, None, A, None, None, 0, None) == want
    if not ok:  # with one too: nothing is launched
        assert lib.moe_decode_ffn(desc, A, A, A, None, *[A] * 6, None, A, None, A, 1 << 40,
                                  None) == want


def test_other_weights_keep_their_widths(lib):  # noqa: F811
    assert lib.moe_grouped_ffn_workspace(ctypes.byref(_desc(T=1, k=1, d=MOST + 128, w=0))) > 0

"""The workspace of the single-token call holds h twice: two bf16 numbers for
each of its values."""
import ctypes

import pytest

from routed_expert_prefill_amd import _lib
from test_abi_operators_cpu import A, _desc, lib  # noqa: F401


@pytest.mark.parametrize("T,k,f", [(1, 6, 256), (2, 6, 256), (16, 4, 2048), (64, 1, 128)])
def test_two_planes(lib, T, k, f):  # noqa: F811
    desc = ctypes.byref(_desc(T=T, k=k, f=f))
    need = lib.moe_decode_ffn_workspace(desc)
    assert need >= T * k * f * 4

    def call(ws_bytes):
        p = [A, A, A, 0, A, A, A, A, A, A, 0, A, 0]
        return lib.moe_decode_ffn(desc, *[v or None for v in p], A, ws_bytes, None)

    assert call(need // 2) == _lib.MOE_EWORKSPACE  # one plane, rounded up
    assert call(need - 1) == _lib.MOE_EWORKSPACE

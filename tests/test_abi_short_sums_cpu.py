"""The type of a dense result with the flag for short sums, on the host: fp32 results
take none (no call here passes validation)."""
import pytest

from routed_expert_prefill_amd import _lib
from test_abi_dense_cpu import A, UNSUP, WS, lib  # noqa: F401

BF16, F32, SHORT = _lib.MOE_DT_BF16, _lib.MOE_DT_F32, _lib.MOE_SHORT_SUMS


@pytest.mark.parametrize("kind,status", [(BF16, WS), (F32, WS), (BF16 | SHORT, WS), (F32 | SHORT, UNSUP),
                                         (2, UNSUP), (2 | SHORT, UNSUP), (SHORT << 1, UNSUP), (-1, UNSUP)])
def test_types_of_results(lib, kind, status):  # noqa: F811
    # a type that is known gets as far as the missing workspace
    assert lib.moe_matmul_fp8(A, None, 4, 100, 256, A, A, A, kind, None, 0, None) == status
    assert lib.moe_shared_ffn(A, None, 4, 256, 128, *[A] * 7, kind, None, 0, None) == status

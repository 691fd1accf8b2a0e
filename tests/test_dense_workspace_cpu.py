"""The workspaces of the dense operators grow with the rows: one for the most serves fewer."""
import os

import pytest

from routed_expert_prefill_amd import _lib


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return _lib.load()


@pytest.mark.parametrize("d,f", [(128, 128), (256, 1152), (640, 1280), (4096, 2048), (16384, 128)])
def test_sizes_grow_with_the_rows(lib, d, f):
    rows = sorted({*range(1, 70), *(1 << i for i in range(18)), *((1 << i) + 1 for i in range(18)), 401, 777, 2049, 3000})
    for query in (lambda T: lib.moe_shared_ffn_workspace(T, d, f), lambda T: lib.moe_matmul_fp8_workspace(T, f, d)):
        sizes = [query(T) for T in rows]
        assert sizes[0] > 0 and sizes == sorted(sizes)
        # what is kept there at the most: codes and scales of the rows, and of h with h in fp32
        assert sizes[-1] <= rows[-1] * (d + d // 32 + f + f // 32 + 4 * f) + 5 * 256

"""The extension module of the short Python calls: it leaves everything but a
good call on the GPU to the Python code, and raises nothing itself."""
import pytest

import routed_expert_prefill_amd as rep


def _module():
    try:
        native = rep._native()
    except rep.LibraryNotBuilt:
        pytest.skip("library not built")
    if native is None:
        pytest.skip("extension module not built")
    return native


def test_leaves_other_calls_to_python():
    import torch

    native = _module()
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    tail = [None] * 5 + [True, True, 0, 0]
    for args in ((), (1,), (x, x[0], 1e-6, *tail), (x, x[0], "eps", *tail), (None, None, 1e-6, *tail),
                 (x, x[0], 1e-6, x, None, None, None, None, 1, True, 0, 0),
                 (x, x[0], 1e-6, *([None] * 5), True, True, "device", 0)):
        assert native.add_rmsnorm(*args) is None
    for args in ((), [x] * 13 + [0, 0], [None] * 13 + [0, 0], [3] * 15, [x] * 13 + [0, "stream"]):
        assert native.decode_ffn(*args) is None
    with pytest.raises(TypeError):
        native.bind(1)


def test_refusals_are_the_python_code_s():
    import torch

    _module()
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        rep.add_rmsnorm(x, x[0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        rep.add_rmsnorm(None, None)
    with pytest.raises(TypeError, match="torch.Tensor"):
        rep.decode_ffn(*[None] * 10, out=x, workspace=x)

"""A status of the launch itself ends a call of expert selection, block
quantisation, an 8-bit product or the shared expert: nothing runs a second time.
A refusal of the argument checks may be asked for again.  Stubs stand for the
library's entry points and for tensors of a GPU."""
import ctypes

import pytest
import torch

import routed_expert_prefill_amd as rep
from routed_expert_prefill_amd import _lib
from test_launch_status_cpu import _on_gpu

vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
TYPES = {
    "moe_route_select": ctypes.CFUNCTYPE(i32, vp, vp, vp, vp, vp, vp),
    "moe_quant_blocks_fp8": ctypes.CFUNCTYPE(i32, vp, i32, i32, i32, vp, vp, vp),
    "moe_matmul_fp8_workspace": ctypes.CFUNCTYPE(sz, i32, i32, i32),
    "moe_matmul_fp8": ctypes.CFUNCTYPE(i32, vp, vp, i32, i32, i32, vp, vp, vp, i32, vp, sz, vp),
    "moe_shared_ffn_workspace": ctypes.CFUNCTYPE(sz, i32, i32, i32),
    "moe_shared_ffn": ctypes.CFUNCTYPE(i32, vp, vp, i32, i32, i32, *[vp] * 7, i32, vp, sz, vp),
}
NAMES = list(TYPES)


class _Lib:
    def __init__(self, lib, **fakes):
        self._lib = lib
        self.__dict__.update(fakes)

    def __getattr__(self, name):
        return getattr(self._lib, name)


@pytest.fixture
def entries(monkeypatch):
    try:
        native = rep._native()
    except rep.LibraryNotBuilt:
        pytest.skip("library not built")
    if native is None:
        pytest.skip("extension module not built")
    lib = _lib.load()
    calls, status = [], [_lib.MOE_EHIP]

    def stub(name):
        if name.endswith("workspace"):
            return getattr(lib, name)

        def f(*args):
            calls.append(name)
            return status[0]

        return f

    fakes = {n: stub(n) for n in NAMES}
    held = [TYPES[n](fakes[n]) for n in NAMES]
    native.bind_dense(*(ctypes.cast(f, vp).value for f in held))
    fake = _Lib(lib, **fakes)
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(_lib, "status_string", lambda code: lib.moe_status_string(code).decode())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    yield calls, status, native
    native.bind_dense(*(ctypes.cast(getattr(lib, n), vp).value for n in NAMES))


def _call(name):
    u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
    z = lambda *shape, dtype=f32: torch.zeros(*shape, dtype=dtype)  # noqa: E731
    if name == "moe_route_select":
        host = [z(2, 8), z(2, 3, dtype=torch.int32), z(2, 3)]
        t = [_on_gpu(h) for h in host]
        return rep.route_select(t[0], 3, topk_ids=t[1], topk_w=t[2]), tuple(t[1:]), host
    if name == "moe_quant_blocks_fp8":
        host = [z(2, 128, dtype=bf), z(2, 128, dtype=u8), z(2, 1)]
        t = [_on_gpu(h) for h in host]
        return rep.quant_blocks_fp8(t[0], q=t[1], s=t[2]), tuple(t[1:]), host
    room = z(1 << 16, dtype=u8)
    if name == "moe_matmul_fp8":
        host = [z(2, 128, dtype=bf), z(8, 128, dtype=u8), z(1, 1), z(2, 8), room]
        t = [_on_gpu(h) for h in host]
        return rep.matmul_fp8(t[0], t[1], t[2], out=t[3], workspace=t[4]), t[3], host
    host = [z(2, 128, dtype=bf), *[z(128, 128, dtype=u8) for _ in range(3)],
            *[z(1, 1) for _ in range(3)], z(2, 128), room]
    t = [_on_gpu(h) for h in host]
    return rep.shared_ffn(*t[:7], out=t[7], workspace=t[8]), t[7], host


CALLS = [n for n in NAMES if not n.endswith("workspace")]


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_not_run_again(entries, name):
    calls, _, _ = entries
    with pytest.raises(RuntimeError, match=f"{name} failed: MOE_EHIP"):
        _call(name)
    assert calls == [name]


@pytest.mark.parametrize("name", CALLS)
def test_a_good_call_is_run_once_and_gives_its_outputs(entries, name):
    calls, status, _ = entries
    status[0] = _lib.MOE_OK
    got, want, _ = _call(name)
    if isinstance(want, tuple):
        assert type(got) is tuple and all(a is b for a, b in zip(got, want))
    else:
        assert got is want
    assert calls == [name]


@pytest.mark.parametrize("name", CALLS)
def test_a_refused_call_gets_its_status_from_python(entries, name):
    calls, status, _ = entries
    status[0] = _lib.MOE_EALIGN
    with pytest.raises(RuntimeError, match="MOE_EALIGN"):
        _call(name)
    assert calls == [name] * 2


def test_the_module_leaves_other_calls_to_python(entries):
    calls, _, native = entries
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    g = _on_gpu(x)
    f = _on_gpu(torch.zeros(2, 128))
    for fn, n in ((native.route_select, 13), (native.quant_blocks_fp8, 5), (native.matmul_fp8, 10),
                  (native.shared_ffn, 14)):
        for args in ((), [x] * n, [None] * n, [g] * (n - 2) + [0, 0], [3] * n, [g] * n):
            assert fn(*args) is None
    select = [f, 3, 1, None, 1, 1, 2, True, 1.0, None, None, 0, 0]
    for at, bad in ((1, 0), (1, 17), (1, 1 << 40), (1, 3.0), (2, None), (4, "1"), (7, 1), (8, 1), (0, x),
                    (3, f), (9, f), (11, "0")):
        assert native.route_select(*[bad if i == at else v for i, v in enumerate(select)]) is None
    assert calls == []
    with pytest.raises(TypeError):
        native.bind_dense(1)


def test_refusals_are_the_python_code_s():
    try:
        rep._native()
    except rep.LibraryNotBuilt:
        pytest.skip("library not built")
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    for call in (lambda: rep.route_select(x, 2), lambda: rep.quant_blocks_fp8(x),
                 lambda: rep.matmul_fp8(x, x, x), lambda: rep.matmul_fp8((x, x), x, x),
                 lambda: rep.shared_ffn(x, *[x] * 6)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: rep.route_select(None, 2), lambda: rep.quant_blocks_fp8(3),
                 lambda: rep.matmul_fp8([x], x, x), lambda: rep.shared_ffn(None, *[x] * 6)):
        with pytest.raises(TypeError, match="torch.Tensor"):
            call()

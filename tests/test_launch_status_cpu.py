"""A status of the launch itself ends a call: nothing runs a second time, since
the first may have run (an addition in place would then count twice).  Stubs
stand for the library's entry points and for tensors of a GPU."""
import ctypes

import pytest
import torch

import routed_expert_prefill_amd as rep
from routed_expert_prefill_amd import _lib

vp, i32 = ctypes.c_void_p, ctypes.c_int
NORM = ctypes.CFUNCTYPE(i32, vp, i32, vp, vp, i32, vp, i32, ctypes.c_float, i32, i32, vp, vp, vp, vp)
DECODE = ctypes.CFUNCTYPE(i32, *[vp] * 15, ctypes.c_size_t, vp)


def _on_gpu(t):
    """A tensor that says it lies on cuda:0, over t's memory."""
    storage = torch._C._construct_storage_from_data_pointer(t.data_ptr(), torch.device("cuda:0"),
                                                            t.nbytes)
    return torch._C._construct_CUDA_Tensor_From_Storage_And_Metadata(
        dict(size=t.shape, stride=t.stride(), dtype=t.dtype, device=torch.device("cuda:0"),
             storage_offset=0), storage)


class _Lib:
    """The library with two entry points replaced."""

    def __init__(self, lib, norm, decode):
        self._lib, self.moe_add_rmsnorm, self.moe_decode_ffn = lib, norm, decode

    def __getattr__(self, name):
        return getattr(self._lib, name)


@pytest.fixture
def entries(monkeypatch):
    """Both ways into the library lead to stubs; status is what they return."""
    try:
        native = rep._native()
    except rep.LibraryNotBuilt:
        pytest.skip("library not built")
    if native is None:
        pytest.skip("extension module not built")
    lib = _lib.load()
    calls, status = [], [_lib.MOE_EHIP]

    def stub(*args):
        calls.append(args)
        return status[0]

    norm, decode = NORM(stub), DECODE(stub)
    native.bind(ctypes.cast(norm, vp).value, ctypes.cast(decode, vp).value)
    fake = _Lib(lib, stub, stub)
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(_lib, "status_string", lambda code: lib.moe_status_string(code).decode())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    yield calls, status
    native.bind(*(ctypes.cast(f, vp).value for f in (lib.moe_add_rmsnorm, lib.moe_decode_ffn)))


def _norm():
    """One call in place, every output given."""
    host = [torch.zeros(4, 8, dtype=torch.bfloat16) for _ in range(3)] + [
        torch.ones(8, dtype=torch.bfloat16)]
    x, r, y, w = (_on_gpu(t) for t in host)
    return rep.add_rmsnorm(x, w, residual=r, residual_out=r, y=y), (y, r, None, None), host


def _decode():
    host = [torch.zeros(1, 128, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32),
            torch.zeros(1, 1), torch.ones(1, 1, dtype=torch.uint8),
            *[torch.zeros(1, 128, 64, dtype=torch.uint8) for _ in range(3)],
            *[torch.zeros(1, 128, 4, dtype=torch.uint8) for _ in range(3)],
            torch.zeros(1, 128), torch.zeros(4096, dtype=torch.uint8)]
    t = [_on_gpu(h) for h in host]
    return rep.decode_ffn(*t[:10], out=t[10], workspace=t[11]), t[10], host


@pytest.mark.parametrize("call,name", [(_norm, "moe_add_rmsnorm"), (_decode, "moe_decode_ffn")])
def test_a_failed_launch_is_not_run_again(entries, call, name):
    calls, _ = entries
    with pytest.raises(RuntimeError, match=f"{name} failed: MOE_EHIP"):
        call()
    assert len(calls) == 1


def test_a_good_call_is_run_once(entries):
    calls, status = entries
    status[0] = _lib.MOE_OK
    got, want, _ = _norm()
    assert all(a is b for a, b in zip(got, want)) and len(calls) == 1
    got, want, _ = _decode()
    assert got is want and len(calls) == 2


@pytest.mark.parametrize("call", [_norm, _decode])
def test_a_refused_call_gets_its_status_from_python(entries, call):
    """The checks refuse ahead of any launch, so Python may ask again."""
    calls, status = entries
    status[0] = _lib.MOE_EALIGN
    with pytest.raises(RuntimeError, match="MOE_EALIGN"):
        call()
    assert len(calls) == 2

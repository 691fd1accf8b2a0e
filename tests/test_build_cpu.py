"""Building where the extension module for short calls cannot be built."""
import os
import sys

import pytest

from routed_expert_prefill_amd import build as B


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """build() with its products under tmp_path and only the C++ part compiled:
    the kernels' objects and the link are stubs."""
    lib, mod = str(tmp_path / "lib.so"), str(tmp_path / "_binding.so")
    monkeypatch.setattr(B, "LIB", lib)
    monkeypatch.setattr(B, "BINDING", mod)
    monkeypatch.setattr(B, "hipcc", lambda: "hipcc")
    real = B._run

    def run(cmd):
        if cmd[0] != "hipcc":
            return real(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            return ""

    monkeypatch.setattr(B, "_run", run)
    return lambda: B.build(out=lib, build_dir=str(tmp_path / "o")), lib, mod


def _without(what, monkeypatch):
    if what == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises
    elif what == "headers":
        monkeypatch.setattr(B, "ROOT", os.path.join(B.ROOT, "nowhere"))  # moe_prefill.h not found
    else:
        monkeypatch.setattr(B.shutil, "which", lambda name: "/nowhere/" + name)


@pytest.mark.parametrize("what", ["torch", "headers", "compiler"])
def test_the_library_is_built_without_the_module(elsewhere, monkeypatch, capsys, what):
    build, lib, mod = elsewhere
    with open(mod, "w") as fh:
        fh.write("of older sources")
    _without(what, monkeypatch)
    assert build() == lib and os.path.exists(lib)
    assert not os.path.exists(mod)
    assert "without the extension module" in capsys.readouterr().err


def test_a_kernel_that_does_not_compile_still_fails(elsewhere, monkeypatch):
    build, lib, _ = elsewhere

    def fails(cmd):
        raise RuntimeError("build failed")

    monkeypatch.setattr(B, "_run", fails)
    with pytest.raises(RuntimeError):
        build()

"""What build() makes and in which order, with the compilers replaced by a
function that writes their outputs."""
from __future__ import annotations

import os
import subprocess
import sys
import types

import pytest

from w4a4_int4_quantized_b200 import build


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Runs of the compilers, in order; `fails` holds the names of those that fail."""
    ran, fails = [], set()

    def run(cmd, **kw):
        ran.append(cmd[0])
        if cmd[0] not in fails:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=int(cmd[0] in fails), stdout="", stderr="")

    monkeypatch.setattr(subprocess, "run", run)
    for name, path in (("LIB", "libw4a4.so"), ("BUILD", "objects"), ("HERE", "")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setenv("CXX", "the-host-compiler")
    return ran, fails


def test_library_is_there_where_the_marshalling_module_cannot_be_built(compilers):
    ran, fails = compilers
    fails.add("the-host-compiler")
    with pytest.raises(RuntimeError, match="the-host-compiler failed"):
        build.build()
    assert os.path.exists(build.LIB) and ran[-1] == "the-host-compiler"


def test_library_without_torch(compilers, monkeypatch):
    ran, _ = compilers
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert "the-host-compiler" not in ran


def test_marshalling_module_is_built_for_the_running_torch(compilers, monkeypatch):
    import torch
    ran, _ = compilers
    build.build()
    first = build.calls_path()
    assert os.path.exists(first) and ran.count("the-host-compiler") == 1
    build.build()
    assert ran.count("the-host-compiler") == 1               # nothing changed
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert build.calls_path() != first and not os.path.exists(build.calls_path())
    build.build()
    assert os.path.exists(build.calls_path()) and ran.count("the-host-compiler") == 2


def test_binding_refuses_a_module_built_for_another_torch(monkeypatch):
    import torch

    import w4a4_int4_quantized_b200 as w4
    build.build()
    monkeypatch.setattr(torch, "__version__", "99.0")
    monkeypatch.setattr(w4, "_calls", None)
    with pytest.raises(w4.W4A4Error) as e:
        w4.w8a8_silu_mul_quantize(torch.zeros(2, 64), torch.zeros(2, 64))
    assert e.value.status == 4 and "not built" in str(e.value.__cause__)

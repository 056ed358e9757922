"""When the build compiles again."""
import os
import shutil
import subprocess

import pytest


@pytest.fixture
def b(monkeypatch, tmp_path):
    """The build with its module in a scratch folder and the compiler's calls counted."""
    from input_adaptive_reduced_rmm_b200 import build

    build.build()
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "OBJ", str(tmp_path))
    if hasattr(build, "BINDING_FOR"):
        monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "_binding.for"))
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        shutil.copy(build.BINDING_SRC, cmd[cmd.index("-o") + 1])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    build.calls = calls
    yield build
    del build.calls


def test_the_module_is_compiled_once(b):
    for n in (1, 1, 1):
        b._build_binding(False)
        assert len(b.calls) == n
    os.utime(b.BINDING, (0, 0))  # older than its source
    b._build_binding(False)
    assert len(b.calls) == 2


@pytest.mark.parametrize("what", ["torch", "python"])
def test_the_module_is_compiled_again_for_another_torch_or_python(b, monkeypatch, what):
    """It uses their C++ and C interfaces: an old build beside new ones fails to load, or worse."""
    import sys

    import torch

    b._build_binding(False)
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    else:
        monkeypatch.setattr(sys, "hexversion", sys.hexversion + 0x10000)
    b._build_binding(False)
    assert len(b.calls) == 2
    b._build_binding(False)
    assert len(b.calls) == 2


def test_a_module_of_unknown_origin_is_compiled_again(b):
    shutil.copy(b.BINDING_SRC, b.BINDING)
    b._build_binding(False)
    assert len(b.calls) == 1

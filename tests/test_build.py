"""The build's commands (none of them is run): with torch and without."""
from __future__ import annotations

import os
import sys

import pytest


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """build.build() with its commands recorded and their outputs made empty, into tmp_path."""
    from implicit_gemm_convolution_amd import build

    ran = []

    def check_call(cmd, **_):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libigc.so"))
    monkeypatch.setattr(build, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))

    def run():
        assert build.build() == str(tmp_path / "libigc.so")
        return ran, sorted(os.listdir(tmp_path))

    return run


def test_build_makes_the_library_and_the_extension(commands):
    ran, files = commands()
    assert files == ["_marshal.so", "libigc.so"] and any("marshal.cpp" in a for c in ran for a in c)


def test_build_without_torch_makes_the_library(commands, monkeypatch):
    for name in [n for n in sys.modules if n == "torch" or n.startswith("torch.utils.cpp_extension")]:
        monkeypatch.delitem(sys.modules, name)
    monkeypatch.setitem(sys.modules, "torch", None)  # (import torch raises ImportError)
    ran, files = commands()
    assert files == ["libigc.so"] and not any("marshal.cpp" in a for c in ran for a in c)
    assert len(ran) > 10

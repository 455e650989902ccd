"""What building rests on: the C library needs nvcc alone, the marshalling module fits the PyTorch it is loaded beside."""
import importlib.util
import os
import subprocess

import pytest
import torch

from reduction_rdx_sum_gb300 import abi, build


@pytest.fixture
def compiles(monkeypatch, tmp_path):
    """The commands that build.py runs, which make an empty file instead of a library."""
    commands = []

    def run(cmd, **kwargs):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "librdx.so"))
    return commands


def marshal_compiles(commands):
    return sum(any(str(word).endswith("marshal.cpp") for word in cmd) for cmd in commands)


def test_the_library_builds_without_pytorch(compiles, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build(force=True, out=build.LIB) == build.LIB and os.path.exists(build.LIB)
    assert marshal_compiles(compiles) == 0 and not os.path.exists(build.MARSHAL)
    with pytest.raises(RuntimeError, match="PyTorch"):
        build.build_marshal()


def test_builds_into_another_path_are_the_library_alone(compiles, tmp_path):
    build.build(defines=["-DRDX_DEBUG=1"], out=str(tmp_path / "checked.so"))
    assert compiles and marshal_compiles(compiles) == 0
    build.build(force=True, out=build.LIB)
    assert marshal_compiles(compiles) == 1

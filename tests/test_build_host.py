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


def test_the_module_is_rebuilt_for_another_pytorch(compiles, monkeypatch):
    build.build_marshal()
    build.build_marshal()
    assert marshal_compiles(compiles) == 1  # up to date
    monkeypatch.setattr(build, "torch_version", lambda: "0.0.1")
    build.build_marshal()
    build.build_marshal()
    assert marshal_compiles(compiles) == 2


def test_a_module_of_another_pytorch_is_not_used(monkeypatch):
    build.build()
    assert build.torch_version() == torch.__version__
    monkeypatch.setattr(abi, "_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="0.0.1"):
        abi._marshal()
    monkeypatch.undo()
    assert abi._marshal().torch_version == torch.__version__

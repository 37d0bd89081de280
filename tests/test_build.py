"""The commands that the build runs (CPU; nothing is compiled here)."""
import sys

import pytest

from sparse_moe_layer_smoe_b200 import build


@pytest.fixture
def commands(monkeypatch):
    run = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: run.append(cmd))
    return run


def test_the_native_module_uses_the_cuda_that_torch_found(commands, monkeypatch):
    from torch.utils import cpp_extension
    monkeypatch.setattr(cpp_extension, "CUDA_HOME", "/opt/some-cuda")
    build.build()
    assert len(commands) == 2 and commands[0][0] == "nvcc"
    includes = [a for a in commands[1] if a.startswith("-I")]
    assert "-I/opt/some-cuda/include" in includes and "-I/usr/local/cuda/include" not in includes


def test_the_library_is_built_without_torch(commands, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert len(commands) == 1 and commands[0][0] == "nvcc"

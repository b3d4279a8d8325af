"""What the build makes of a host that lacks a part: compilers are stand-ins that
write their output file, or fail."""

import os
import sys

import pytest

from exact_attention_64_gb300 import build as b


class _Tools:
    def __init__(self, tmp, monkeypatch):
        self.ran, self.broken = [], ()
        monkeypatch.setattr(b, "BUILD", tmp / "_build")
        monkeypatch.setattr(b, "LIB", tmp / "libfa2.so")
        monkeypatch.setattr(b, "BINDING", tmp / "_binding.so")
        monkeypatch.setattr(b, "BINDING_FOR", tmp / "_build" / "binding_for.txt")
        if hasattr(b, "BINDING_ERROR"):
            monkeypatch.setattr(b, "BINDING_ERROR", tmp / "_build" / "binding_error.txt")
        monkeypatch.setattr(b, "_run", self.run)

    def run(self, cmd, what, verbose):
        tool = os.path.basename(cmd[0])
        if tool in self.broken:
            raise RuntimeError(f"{what}: {tool} is broken")
        self.ran.append(tool)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass


@pytest.fixture
def tools(tmp_path, monkeypatch):
    monkeypatch.delenv("CXX", raising=False)
    return _Tools(tmp_path, monkeypatch)


def test_everything_then_nothing(tools):
    assert b.needs_build()
    assert b.build() == b.LIB
    assert b.LIB.exists() and b.BINDING.exists() and not b.needs_build()
    n = len(tools.ran)
    assert n == len(b._sources()) + 3
    b.build()
    assert len(tools.ran) == n


def test_a_host_without_a_python_toolchain_gets_the_library(tools):
    tools.broken = ("g++",)
    with pytest.warns(RuntimeWarning, match="g[+][+] is broken"):
        assert b.build() == b.LIB
    assert b.LIB.exists() and not b.BINDING.exists()
    n = len(tools.ran)
    with pytest.warns(RuntimeWarning):
        b.build()  # only the binding is tried again
    assert len(tools.ran) == n
    tools.broken = ()
    b.build()
    assert b.BINDING.exists() and tools.ran[n:] == ["g++", "g++"] and not b.needs_build()


def test_a_host_without_pytorch_gets_the_library(tools, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert b.needs_build()
    assert b.build() == b.LIB
    assert b.LIB.exists() and not b.BINDING.exists() and "g++" not in tools.ran
    assert not b.needs_build()


def test_another_pytorch_rebuilds_only_the_binding(tools):
    b.build()
    n = len(tools.ran)
    b.BINDING_FOR.write_text("another one")
    assert b.needs_build()
    b.build()
    assert tools.ran[n:] == ["g++", "g++"]


def test_a_broken_cuda_compiler_raises(tools):
    tools.broken = ("nvcc",)
    with pytest.raises(RuntimeError, match="nvcc is broken"):
        b.build()
    assert not b.LIB.exists()

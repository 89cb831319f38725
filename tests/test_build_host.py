"""What the build does where parts of it are missing or have changed, with the compilers replaced by a stand-in (no GPU and
no compiler needed)."""
import os
import subprocess

import pytest

from context_causal_attention_gb300 import build as B


class Compiler:
    """Takes subprocess.run's place: writes the outputs that a command names; `fails` says which commands do not."""

    def __init__(self):
        self.commands, self.fails = [], lambda cmd: False

    def run(self, cmd, **kw):
        self.commands.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        if self.fails(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "it does not compile")
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def sources(self):
        got = sorted(os.path.basename(c[c.index("-c") + 1]) for c in self.commands if "-c" in c)
        self.commands = []
        return got


ALL = sorted(B.SOURCES + ["bind.cpp"])


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    c = Compiler()
    monkeypatch.setattr(B.subprocess, "run", c.run)
    monkeypatch.setattr(B, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(B, "OUT", str(tmp_path))
    for name, file in (("LIB", "libcpattn.so"), ("BIND", "_cpbind.so"), ("TAG", "_cpbind.tag")):
        monkeypatch.setattr(B, name, str(tmp_path / file), raising=False)
    monkeypatch.setattr(B.shutil, "which", lambda exe: "/usr/bin/" + exe)
    monkeypatch.setattr(B.os.path, "exists", exists_with_headers)
    return c


real_exists = os.path.exists


def exists_with_headers(path):
    return real_exists(path) or str(path).endswith((".h", "nvcc"))


def test_all_once_and_then_nothing(compiler):
    assert B.build() == B.LIB and compiler.sources() == ALL
    assert os.path.getsize(B.LIB) and os.path.getsize(B.BIND)
    assert B.build() == B.LIB and compiler.commands == []
    assert B.build(force=True) == B.LIB and compiler.sources() == ALL


@pytest.mark.parametrize("lacks", ["Python.h", "python_variable.h", "g++"])
def test_the_library_without_what_the_module_needs(compiler, monkeypatch, capsys, lacks):
    """nvcc alone builds the library, as it did before there was a module; an old module does not stay."""
    B.build()
    compiler.commands = []
    if lacks == "g++":
        monkeypatch.setattr(B.shutil, "which", lambda exe: None if exe == "g++" else "/usr/bin/" + exe)
    else:
        monkeypatch.setattr(B.os.path, "exists", lambda p: not str(p).endswith(lacks) and exists_with_headers(p))
    assert B.build(force=True) == B.LIB and compiler.sources() == sorted(B.SOURCES)
    assert os.path.getsize(B.LIB) and not real_exists(B.BIND)
    assert lacks in capsys.readouterr().err


def test_the_library_stands_where_the_module_does_not_compile(compiler):
    compiler.fails = lambda cmd: cmd[-3].endswith("bind.cpp") or any(str(x).endswith("bind.cpp") for x in cmd)
    with pytest.raises(RuntimeError, match="bind.cpp"):
        B.build()
    assert os.path.getsize(B.LIB) and not real_exists(B.BIND)
    compiler.fails = lambda cmd: False
    compiler.commands = []
    assert B.build() == B.LIB and compiler.sources() == ["bind.cpp"]  # and the next build makes it alone


def test_another_torch_makes_another_module(compiler, monkeypatch):
    B.build()
    compiler.commands = []
    monkeypatch.setattr(B.importlib.metadata, "version", lambda name: "9.9.9")
    assert B.build() == B.LIB and compiler.sources() == ["bind.cpp"]
    assert B.build() == B.LIB and compiler.commands == []


def test_a_cuda_source_that_does_not_compile_is_told(compiler):
    compiler.fails = lambda cmd: any(str(x).endswith("tree.cu") for x in cmd)
    with pytest.raises(RuntimeError, match="tree.cu"):
        B.build()
    assert not real_exists(B.LIB)

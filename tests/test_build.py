"""What the build makes, in which order, and when again, with the compilers replaced
by a stand-in that writes the file it is asked for."""

import os
import subprocess
import sys

import pytest

from weight_gated_mlp_b200 import _build


class Compiler:
    """Stands in for subprocess.run: notes what is made and writes it, or fails."""

    def __init__(self):
        self.made, self.failing = [], None

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).removesuffix(".tmp")
        self.made.append(name)
        if name == self.failing:
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        with open(out, "w") as f:
            f.write("x")
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    c = Compiler()
    monkeypatch.setattr(_build.subprocess, "run", c)
    monkeypatch.setattr(_build, "nvcc_path", lambda: "/usr/local/cuda/bin/nvcc")
    for name, file in (("LIB", "libittt.so"), ("MARSHAL", "_marshal.so")):
        monkeypatch.setattr(_build, name, str(tmp_path / file))
    return c


def test_both_once(compiler):
    assert _build.build() == _build.LIB
    assert sorted(compiler.made) == ["_marshal.so", "libittt.so"]
    _build.build()
    assert len(compiler.made) == 2
    _build.build(force=True)
    assert len(compiler.made) == 4


def test_the_library_needs_no_torch(compiler, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)      # as if it were not installed
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB)
    assert compiler.made == ["libittt.so"]
    assert "torch" in capsys.readouterr().err


def test_the_library_needs_no_python_headers(compiler, monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    assert _build.build() == _build.LIB
    assert compiler.made == ["libittt.so"]
    assert "header" in capsys.readouterr().err


def test_a_module_that_does_not_compile_is_an_error_behind_the_library(compiler):
    compiler.failing = "_marshal.so"
    with pytest.raises(RuntimeError, match=r"g\+\+ failed"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.MARSHAL)


def test_another_torch_makes_the_module_again(compiler, monkeypatch):
    _build.build()
    monkeypatch.setattr(_build, "marshal_key", lambda: "another torch")
    _build.build()
    _build.build()
    assert compiler.made == ["libittt.so", "_marshal.so", "_marshal.so"]

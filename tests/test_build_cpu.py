"""What the build makes and for whom: the CUDA library for every caller, the binding for one Python and one
PyTorch. The compilers are replaced by ones that write a file."""
import importlib.metadata
import os
import subprocess
import sys

import pytest

import paged_kv_decode_gqa_b200 as pkv
from paged_kv_decode_gqa_b200 import build as b


@pytest.fixture
def runs(tmp_path, monkeypatch):
    """The commands that ran; outputs go to an empty folder."""
    commands = []

    def run(cmd, check=False, **kw):
        commands.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0)

    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING_DIR", str(tmp_path))
    monkeypatch.setattr(b.subprocess, "run", run)
    return commands


def compilers(commands):
    return [os.path.basename(c[0]) for c in commands]


def test_both_are_built_and_then_up_to_date(runs):
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.binding_path())
    assert compilers(runs) == ["nvcc", os.path.basename(os.environ.get("CXX", "g++"))]
    b.build()
    assert len(runs) == 2


def test_the_library_needs_no_pytorch(runs, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)                # an import of it raises ImportError
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert compilers(runs) == ["nvcc"]
    assert "binding" in capsys.readouterr().err
    with pytest.raises(ImportError):
        b.build_binding()


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, "g++")])
def test_the_library_needs_no_cpp_compiler(runs, monkeypatch, capsys, error):
    fake = b.subprocess.run

    def run(cmd, **kw):
        if os.path.basename(cmd[0]) != "nvcc":
            raise error
        return fake(cmd, **kw)

    monkeypatch.setattr(b.subprocess, "run", run)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.binding_path())
    assert "binding" in capsys.readouterr().err


def test_a_library_that_does_not_compile_is_an_error(runs, monkeypatch):
    def run(cmd, **kw):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.raises(subprocess.CalledProcessError):
        b.build()


def test_the_binding_is_built_anew_for_another_pytorch(runs, monkeypatch):
    b.build()
    first, n = b.binding_path(), len(runs)
    real = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9" if name == "torch" else real(name))
    assert b.binding_path() != first and not os.path.exists(b.binding_path())
    with pytest.raises(ImportError, match="not built"):            # the one of the other PyTorch is not loaded
        pkv._load_binding()
    b.build()
    assert os.path.exists(b.binding_path()) and len(runs) == n + 1
    with open(first):                                              # (which may be used elsewhere still)
        pass


def test_the_name_tells_the_python(monkeypatch):
    name = os.path.basename(b.binding_path())
    assert sys.implementation.cache_tag.replace("cpython-", "") in name
    assert importlib.metadata.version("torch") in name

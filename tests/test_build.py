"""What is built when, with the compilers replaced by a recorder: libpkv.so does not depend on the binding, and the binding
is built again for another torch.  No GPU."""
import os
import subprocess
import types

import pytest
import torch

import paged_kv_cache_175_gb300 as pkv
from paged_kv_cache_175_gb300 import _build


class Compilers:
    """Stands for subprocess.run: writes each command's output file, or fails it."""

    def __init__(self):
        self.ran, self.fails = [], lambda cmd: None

    def __call__(self, cmd, **kw):
        error = self.fails(cmd)
        if error is FileNotFoundError:
            raise FileNotFoundError(cmd[0])
        if error:
            return subprocess.CompletedProcess(cmd, 1, "", error)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        self.ran.append(os.path.basename(out).removesuffix(".tmp"))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def take(self):
        got, self.ran = sorted(self.ran), []
        return got


@pytest.fixture
def tools(tmp_path, monkeypatch):
    c = Compilers()
    monkeypatch.setattr(_build, "subprocess", types.SimpleNamespace(run=c))
    monkeypatch.setattr(_build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(_build, "CALLS_KEY", str(tmp_path / "obj" / "calls.key"))
    return c


LIB_OUT = sorted([os.path.splitext(s)[0] + ".o" for s in _build.SOURCES] + ["libpkv.so"])
CALLS_OUT = ["_calls.so", "calls.o"]


def test_builds_both_once(tools):
    assert _build.build_library() == _build.LIB
    assert tools.take() == sorted(LIB_OUT + CALLS_OUT) and _build.calls_current()
    _build.build_library()
    assert tools.take() == []
    _build.build_library(force=True)
    assert tools.take() == sorted(LIB_OUT + CALLS_OUT)


@pytest.mark.parametrize("what", ["compile", "link", "no g++"])
def test_the_library_is_there_where_the_binding_cannot_be_built(tools, what):
    tools.fails = {"compile": lambda c: "no Python.h" if "calls.cpp" in " ".join(c) else None,
                   "link": lambda c: "no c10_cuda" if "-lc10_cuda" in c else None,
                   "no g++": lambda c: FileNotFoundError if c[0] == "g++" else None}[what]
    with pytest.warns(UserWarning, match="_calls.so was not built"):
        assert _build.build_library() == _build.LIB
    assert os.path.exists(_build.LIB) and "libpkv.so" in tools.take() and not _build.calls_current()
    tools.fails = lambda c: None
    _build.build_library()                                     # later only the binding is missing
    assert tools.take() == CALLS_OUT and _build.calls_current()


def test_the_library_itself_fails_loudly(tools):
    tools.fails = lambda c: "bad" if "evict.cu" in " ".join(c) else None
    with pytest.raises(RuntimeError, match="evict.cu"):
        _build.build_library()
    assert not os.path.exists(_build.LIB)


def test_the_binding_is_built_again_for_another_torch(tools, monkeypatch):
    _build.build_library()
    tools.take()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert not _build.calls_current()
    _build.build_library()
    assert tools.take() == CALLS_OUT and _build.calls_current()


def test_a_binding_of_another_torch_is_not_loaded(tools, monkeypatch):
    _build.build_library()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    monkeypatch.setattr(pkv, "_calls", None)
    with pytest.raises(pkv.PkvError, match="another torch"):
        pkv._native()

"""What build.py builds and when: the C library with and without torch, the
extension for the torch that is installed.  Compilers are replaced by a
function that writes their output files."""
import os
import subprocess
import sys

import pytest

from paged_kv_cache_112_gb300 import build as B


class Compilers:
    def __init__(self):
        self.outputs, self.fail = [], None

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".tmp")[0]
        if name == self.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "broken")
        self.outputs.append(name)
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    c = Compilers()
    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(B, "EXT", str(tmp_path / "_pkv_torch.so"))
    monkeypatch.setattr(B, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(B.subprocess, "run", c)
    return c


def built(c):
    n = [os.path.exists(p) for p in (B.LIB, B.EXT)]
    made, c.outputs = set(c.outputs), []
    return n, made


def test_library_and_extension(compilers):
    assert B.build() == B.LIB
    there, made = built(compilers)
    assert there == [True, True] and {"libpkv.so", "_pkv_torch.so", "pkv_torch.o", "pkv_api.o"} <= made
    B.build()
    assert built(compilers) == ([True, True], set())  # nothing to do
    B.build(force=True)
    assert {"libpkv.so", "_pkv_torch.so"} <= built(compilers)[1]


def test_library_without_torch(compilers, monkeypatch, capsys):
    """The C library needs no torch; the extension is left out, and built once torch is there."""
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)  # import torch raises ImportError
        assert B.build() == B.LIB
        there, made = built(compilers)
        assert there == [True, False] and "libpkv.so" in made and "pkv_torch.o" not in made
        assert "torch" in capsys.readouterr().err
        B.build()
        assert built(compilers) == ([True, False], set())
    B.build()
    assert built(compilers) == ([True, True], {"pkv_torch.o", "_pkv_torch.so"})


def test_library_beside_an_extension_that_does_not_compile(compilers):
    compilers.fail = "pkv_torch.o"
    with pytest.raises(RuntimeError, match="pkv_torch.cpp"):
        B.build()
    assert built(compilers)[0] == [True, False]

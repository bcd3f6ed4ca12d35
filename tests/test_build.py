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


def test_extension_of_another_torch(compilers, monkeypatch):
    """Another installed torch makes the extension stale, whatever the files' times; the library is not."""
    import torch

    B.build()
    built(compilers)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1+other")
        B.build()
        assert built(compilers) == ([True, True], {"pkv_torch.o", "_pkv_torch.so"})
        assert '-DPKV_TORCH_VERSION="0.0.1+other"' in open(os.path.join(B.OUT_DIR, "pkv_torch.o")).read()
        B.build()
        assert built(compilers)[1] == set()
    B.build()
    assert built(compilers)[1] == {"pkv_torch.o", "_pkv_torch.so"}


def test_an_extension_of_another_torch_is_refused(monkeypatch):
    """One that was built before torch changed: the first layer operator says what to do."""
    import torch

    import paged_kv_cache_112_gb300 as pkv
    from paged_kv_cache_112_gb300 import _binding

    try:
        B.build()
    except RuntimeError as e:  # no nvcc on this machine
        pytest.skip(str(e))
    monkeypatch.setattr(_binding, "_EXT", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(pkv.PkvError, match="rebuild"):
        _binding._ext()
    assert _binding._EXT is None

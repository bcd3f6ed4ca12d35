"""Builds libpkv.so in-tree with nvcc for sm_103a (GB300), and beside it the
extension that passes torch tensors to its layer operators (g++).

Each translation unit compiles in parallel; the result links the CUDA runtime
statically, so the library needs only the NVIDIA driver at run time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpkv.so")
EXT = os.path.join(OUT_DIR, "_pkv_torch.so")  # CPython extension over libpkv and torch
EXT_SOURCE = "pkv_torch.cpp"
SOURCES = ["pkv_api.cu", "pkv_cache_ops.cu", "pkv_decode.cu", "pkv_decode_hg.cu", "pkv_decode_balanced.cu",
           "pkv_decode_fp8.cu", "pkv_norm_rope.cu", "pkv_sparse_select.cu", "pkv_sparse_decode.cu", "pkv_api_layer.cu",
           "pkv_static_ws.cu", "pkv_checks.cu", "pkv_block_manager.cpp"]
HEADERS = ["pkv_internal.h", "pkv_device.cuh", "pkv_balanced.cuh", "pkv_fp8.cuh", "pkv_fp8_attention.cuh", os.path.join("..", "..", "include", "pkv.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv")


def _older(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps + [os.path.abspath(__file__)])


def _lib_stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS])


def _ext_stale(version: str) -> bool:
    """Older than its sources, or built for another torch than `version`."""
    if _older(EXT, [os.path.join(CSRC, EXT_SOURCE), os.path.join(ROOT, "include", "pkv.h")]):
        return True
    if not os.path.exists(EXT + ".torch"):
        return True
    with open(EXT + ".torch") as f:
        return f.read() != version


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Builds what is missing, older than its sources or made for another torch.  The library needs no torch:
    where torch does not import, the extension is left out and stderr says so."""
    lib, torch_dirs = force or _lib_stale(), None
    try:
        torch_dirs = _torch_dirs()
    except Exception as e:  # not installed, or installed and broken
        sys.stderr.write(f"{os.path.basename(EXT)} is not built: torch does not import ({e})\n")
    if torch_dirs and not (force or _ext_stale(torch_dirs[2])):
        torch_dirs = None
    if not lib and not torch_dirs:
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext_obj = ex.submit(_compile_ext, torch_dirs) if torch_dirs else None
        if lib:
            _build_lib(nvcc, ex, verbose, ptxas_verbose)
        if ext_obj:
            _link_ext(ext_obj.result(), torch_dirs)
    return LIB


def _build_lib(nvcc: str, ex: ThreadPoolExecutor, verbose: bool, ptxas_verbose: bool) -> None:
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")  # .cpp: host code through nvcc
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _torch_dirs() -> tuple:
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    return os.path.join(root, "include"), os.path.join(root, "lib"), torch.__version__


def _compile_ext(torch_dirs: tuple) -> str:
    inc, _, version = torch_dirs
    obj = os.path.join(OUT_DIR, "pkv_torch.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", os.path.join(ROOT, "include"), "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
           sysconfig.get_paths()["include"], f'-DPKV_TORCH_VERSION="{version}"', "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ext(obj: str, torch_dirs: tuple) -> None:
    """Links against libpkv.so beside it and the installed torch."""
    _, lib, version = torch_dirs
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-l:libpkv.so", "-L", lib, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(EXT + ".torch", "w") as f:
        f.write(version)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))

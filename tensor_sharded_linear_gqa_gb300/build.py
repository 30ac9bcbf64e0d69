"""Builds the in-tree shared library ``libtpgqa.so`` for sm_103a with nvcc.

Each translation unit is compiled in parallel into ``_build/`` and linked into
``tensor_sharded_linear_gqa_gb300/libtpgqa.so`` (static CUDA runtime; the driver
API is reached through cudaGetDriverEntryPointByVersion, so libcuda is not a
link dependency). A stamp records the machine and the source hashes, so a
library built for another machine or from other sources is rebuilt. Beside it
lies ``_describe.so``, an extension module of the Python binding.

Usage: ``python -m tensor_sharded_linear_gqa_gb300.build [--force] [-v]``.
"""
from __future__ import annotations

import hashlib
import importlib.util
import json
import os
import platform
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtpgqa.so")
STAMP = os.path.join(BUILD, "stamp.json")
DESCRIBE = os.path.join(PKG, "_describe.so")  # the binding's extension module

SOURCES = ["plan.cpp", "tp_api.cu", "gemm_tcgen05.cu", "gemm_f32.cu", "combine.cu", "mlp_static.cu", "vocab.cu", "moe.cu", "attention.cu",
           "rmsnorm.cu", "cache_evict.cu", "linear_epilogue.cu", "prefix_attention.cu",
           "rotary.cu", "window_attention.cu", "cache4.cu"]
HEADERS = ["tp_internal.h", "sm100_ptx.cuh", "op_util.h", "split_join.cuh", "describe.c", "describe_torch.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libtpgqa.so")


def _digest() -> str:
    h = hashlib.sha256()
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "tpgqa.h"),
                                                                  os.path.abspath(__file__)]
    for f in files:
        with open(f, "rb") as fh:
            h.update(os.path.basename(f).encode())
            h.update(fh.read())
    return h.hexdigest()


def _python_h() -> str:
    return os.path.join(sysconfig.get_paths()["include"], "Python.h")


def _torch() -> tuple:
    """(version and revision, folder) of the installed torch, without importing it; (None, None) without
    one, or with one that does not say which it is."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None, None
    folder = list(spec.submodule_search_locations)[0]
    try:
        with open(os.path.join(folder, "version.py")) as fh:
            text = fh.read()
    except OSError:
        return None, None
    found = [re.search(rf"^{name}\b[^=\n]*= *['\"]([\w.+-]+)['\"]", text, re.M) for name in ("__version__", "git_version")]
    if None in found:
        return None, None
    return " ".join(m[1] for m in found), folder


def _stamp() -> dict:
    return {"machine": platform.machine(), "digest": _digest(), "python": sysconfig.get_config_var("SOABI"), "torch": _torch()[0]}


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(STAMP):
        return False
    if os.path.exists(_python_h()) and not os.path.exists(DESCRIBE):
        return False
    try:
        with open(STAMP) as fh:
            return json.load(fh) == _stamp()
    except (OSError, ValueError):
        return False


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "c++"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def _compile_describe_torch(verbose: bool) -> list:
    """Compiles what reads torch tensors directly; the objects and libraries to link, none without torch's headers."""
    version, folder = _torch()
    if folder is None or not os.path.exists(os.path.join(folder, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return []
    if not os.path.exists(_python_h()):
        return []
    with open(os.path.join(BUILD, "torch_version.h"), "w") as fh:
        fh.write(f'#define TP_TORCH_VERSION "{version}"\n')
    obj = os.path.join(BUILD, "describe_torch.o")
    cmd = [nvcc(), "-x", "c++", "-std=c++20", "-O2", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", os.path.join(folder, "include"),
           "-I", os.path.dirname(_python_h()), "-c", os.path.join(CSRC, "describe_torch.cpp"), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(f"describe_torch.cpp does not compile against {folder}: tensors are described by way of their attributes\n"
              + r.stderr[-2000:], file=sys.stderr)
        return []
    return [obj, "-L", os.path.join(folder, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]


def _build_describe(torch_parts: list, verbose: bool) -> None:
    """Compiles the extension module that describes tensors; without the interpreter's headers
    there is none, and the binding does without."""
    if not os.path.exists(_python_h()):
        print(f"{_python_h()} is missing: tensors are described by interpreted code", file=sys.stderr)
        return
    obj, tmp = os.path.join(BUILD, "describe.o"), DESCRIBE + ".tmp"
    for cmd in ([nvcc(), "-x", "c", "-O2", "-Xcompiler", "-fPIC", *(["-DTP_WITH_TORCH", "-I", BUILD] if torch_parts else []), "-I", INCLUDE,
                 "-I", os.path.dirname(_python_h()), "-c", os.path.join(CSRC, "describe.c"), "-o", obj],
                [nvcc(), "-cudart", "none", "-shared", obj, *torch_parts, "-o", tmp]):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 and torch_parts:
            print("describe_torch.cpp does not link: tensors are described by way of their attributes\n" + r.stderr[-2000:],
                  file=sys.stderr)
            return _build_describe([], verbose)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on describe.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, DESCRIBE)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles and links libtpgqa.so if it is missing or stale; returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        torch_parts = ex.submit(_compile_describe_torch, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _build_describe(torch_parts.result(), verbose)
    with open(STAMP, "w") as fh:
        json.dump(_stamp(), fh)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

"""Builds libfas.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_host.so (its calls on torch tensors) with the host compiler.

Usage: ``python -m frame_aligned_sparse_gb300.build`` or ``build()``.
Translation units compile in parallel; the shared object lands next to this
file.  Objects go to ``_build/`` (git-ignored).
"""
from __future__ import annotations

import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libfas.so")
HOST_SRC = os.path.join(CSRC, "host", "calls.cpp")
HOST_OUT = os.path.join(PKG, "_host.so")
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
BUILD = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfas.so")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _torch() -> Optional[str]:
    """The installed torch's folder, without importing it (a slow import)."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    folders = list(spec.submodule_search_locations or ()) if spec else []
    return folders[0] if folders else None


def _host_command(torch: str, out: str) -> list:
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    includes = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    return (["g++", HOST_SRC, "-o", out] + ["-I" + i for i in includes] + ["-L" + os.path.join(torch, "lib")] +
            HOST_FLAGS)


def _fingerprint() -> str:
    h = hashlib.sha256()
    files = _sources() + sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh")))
    files += [os.path.join(INCLUDE, "fas.h"), HOST_SRC]
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    h.update(os.uname().machine.encode())
    torch = _torch()
    if torch:
        h.update(" ".join([torch] + HOST_FLAGS).encode())
        version = os.path.join(torch, "version.py")
        if os.path.exists(version):
            with open(version, "rb") as fh:
                h.update(fh.read())
    return h.hexdigest()


_WITHOUT_HOST = " without _host.so"  # in the stamp: it did not compile here


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not up to date and returns libfas.so's path.  _host.so
    only saves time on calls with torch tensors, so it is left out, with a
    warning, where torch or what compiling against it takes is missing (tried
    again when a source or torch changes, or with force)."""
    stamp = os.path.join(BUILD, "stamp")
    fp = _fingerprint()
    torch = _torch()  # without it libfas.so alone: the C boundary needs none
    if not force and os.path.exists(OUT) and os.path.exists(stamp):
        with open(stamp) as fh:
            was = fh.read()
        if was == fp + _WITHOUT_HOST or (was == fp and (not torch or os.path.exists(HOST_OUT))):
            return OUT
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc] + ARCH + FLAGS + ["-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr, file=sys.stderr)
        return obj

    def compile_host() -> bool:
        tmp = HOST_OUT + ".tmp"
        try:
            res = subprocess.run(_host_command(torch, tmp), capture_output=True, text=True)
            failed = f"{res.stdout}\n{res.stderr}" if res.returncode else ""
        except OSError as e:
            failed = str(e)
        if not failed:
            os.replace(tmp, HOST_OUT)
            return True
        if os.path.exists(HOST_OUT):  # of other sources or another torch
            os.remove(HOST_OUT)
        print(f"warning: building without {os.path.basename(HOST_OUT)} (calls on torch tensors take longer): g++ failed "
              f"on {HOST_SRC}:\n{failed[-4000:]}", file=sys.stderr)
        return False

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 1)) as ex:
        host = ex.submit(compile_host) if torch else None
        objs = list(ex.map(compile_one, srcs))
        without = "" if not host or host.result() else _WITHOUT_HOST
    tmp = OUT + ".tmp"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, OUT)
    with open(stamp, "w") as fh:
        fh.write(fp + without)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

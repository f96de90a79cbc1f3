"""Build libpoetx.so (the POET-X layer's C ABI and its sm_100a kernels) in
place, next to this file, with nvcc; `debug=True` builds libpoetx_debug.so,
the same library compiled with -DPOETX_DEBUG (every TMA and bulk copy checked
before it is issued; see csrc/ptx.cuh), loaded instead when the environment
sets POETX_DEBUG=1.  Either build also brings up to date _tensors.so, a Python
extension (host code only) that calls whichever library is loaded."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpoetx.so")
LIB_DEBUG = os.path.join(HERE, "libpoetx_debug.so")
TENSORS = os.path.join(HERE, "_tensors.so")   # csrc/tensors.cpp: the torch side of quantized.py
SOURCES = ["poetx.cu"]


def deps():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))) +
            [os.path.join(ROOT, "include", "poetx.h")])


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps() if os.path.exists(d))


def built_for() -> bytes:
    """What an extension is compiled against, as _tensors.so holds it."""
    import torch
    return f"poetx built for torch {torch.__version__}, {sys.implementation.cache_tag};".encode()


def tensors_up_to_date(src) -> bool:
    if not os.path.exists(TENSORS) or os.path.getmtime(TENSORS) < max(os.path.getmtime(f) for f in src):
        return False
    with open(TENSORS, "rb") as f:
        return built_for() in f.read()


def build_tensors(force: bool = False) -> str:
    """The extension of csrc/tensors.cpp, compiled against the installed torch
    (again when that or Python has changed)."""
    src = [os.path.join(CSRC, "tensors.cpp"), os.path.join(ROOT, "include", "poetx.h")]
    if not force and tensors_up_to_date(src):
        return TENSORS
    import sysconfig

    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = f"{TENSORS}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DPOETX_BUILT_FOR="{built_for().decode()}"', "-I", os.path.join(ROOT, "include"),
           "-I", os.path.join(at, "include"), "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), src[0], "-o", tmp,
           "-L", os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{cmd[0]} failed building {os.path.basename(TENSORS)}")
    os.replace(tmp, TENSORS)
    return TENSORS


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """The library, then the extension; the library alone, which needs nothing
    but nvcc, where torch is not installed."""
    lib = LIB_DEBUG if debug else LIB
    if force or needs_build(lib):
        build_library(lib, verbose, debug)
    try:
        import torch  # noqa: F401
    except ImportError as e:
        sys.stderr.write(f"{os.path.basename(TENSORS)} (the torch functions) not built: {e}\n")
        return lib
    build_tensors(force)
    return lib


def build_library(lib: str, verbose: bool, debug: bool) -> None:
    cmd = [nvcc(), "-std=c++17", "-O3", "-lineinfo", "-gencode", "arch=compute_100a,code=sm_100a",
           "-shared", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-o", lib + ".tmp"] + [os.path.join(CSRC, s) for s in SOURCES] + ["-lcudart"]
    if debug:
        cmd.insert(1, "-DPOETX_DEBUG")
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc failed building {os.path.basename(lib)}")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(lib + ".tmp", lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))

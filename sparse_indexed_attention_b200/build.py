"""Builds libdsa.so (nvcc, sm_100a) and the Python binding's native part
_binding.so (g++, on torch's headers) in-tree.  No GPU needed to build.

    python -m sparse_indexed_attention_b200.build [--force]
"""
from __future__ import annotations

import fcntl
import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdsa.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(PKG, "_binding.built_for")     # the torch and Python that _binding.so was compiled against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
          "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: libdsa.so cannot be built")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [
        BINDING_SRC, os.path.abspath(__file__)]


def target() -> str:
    """The torch and Python whose C++ layouts _binding.so takes from their headers."""
    import sysconfig

    import torch

    return (f"torch {torch.__version__} {torch.version.git_version} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"{sysconfig.get_config_var('SOABI')}\n")


def _newer_input(than: str) -> bool:
    t = os.path.getmtime(than)
    return any(os.path.getmtime(p) > t for p in _inputs())


def library_is_stale() -> bool:
    return not os.path.exists(LIB) or _newer_input(LIB)


def binding_is_stale() -> bool:
    """Also where it was built for another torch or Python: it would read their objects wrongly."""
    if not os.path.exists(BINDING) or not os.path.exists(BUILT_FOR) or _newer_input(BINDING):
        return True
    with open(BUILT_FOR) as f:
        return f.read() != target()


def is_stale() -> bool:
    return library_is_stale() or binding_is_stale()


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)          # concurrent importers build once
        if force or library_is_stale():
            _build_library(verbose)
        if force or binding_is_stale():
            _build_binding()
        return LIB


def _binding_command(out: str) -> list[str]:
    import sysconfig

    import torch

    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found: _binding.so cannot be built")
    inc = [os.path.join(t, "include"), os.path.join(t, "include/torch/csrc/api/include"), os.path.join(cuda, "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    return [cxx, "-O2", "-fPIC", "-shared", "-std=c++17", *(a for d in inc for a in ("-isystem", d)), BINDING_SRC, "-o",
            out, "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-L", PKG, "-l:libdsa.so", "-Wl,-rpath,$ORIGIN"]


def _build_library(verbose: bool) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_binding() -> None:
    tmp = BINDING + ".tmp"
    r = subprocess.run(_binding_command(tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stderr}")
    if os.path.exists(BUILT_FOR):
        os.remove(BUILT_FOR)
    os.replace(tmp, BINDING)
    with open(BUILT_FOR + ".tmp", "w") as f:
        f.write(target())
    os.replace(BUILT_FOR + ".tmp", BUILT_FOR)


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))

"""Builds libcsa.so in-tree with nvcc for sm_103a (no torch extension machinery).

Each .cu file compiles to an object in parallel, then one shared-library link.
The build is skipped when the library is newer than every source and header.
csa_torch, the serving helpers' short way from tensors to the library, is a CPython
extension against torch's headers (no CUDA code of its own), compiled beside it by
build() or on the helpers' first call; they do without where it cannot be had.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libcsa.so")
OBJDIR = os.path.join(PKG, "_build")
BINDING_SRC = os.path.join(CSRC, "csa_torch.cpp")
BINDING = os.path.join(PKG, "csa_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# No --use_fast_math: the kernels need IEEE division/reciprocal and no flush-to-zero.
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcsa")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                               + glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in _deps())


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return None if spec is None else list(spec.submodule_search_locations)[0]


def binding_stale() -> bool:
    if not os.path.exists(BINDING):
        return True
    deps = [BINDING_SRC, os.path.abspath(__file__), os.path.join(_torch_dir(), "version.py")]
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > os.path.getmtime(BINDING) for d in deps if os.path.exists(d))


def build_binding(force: bool = False) -> str:
    """Compile csa_torch.so if missing or stale (it is newer than the torch it was built against); returns its path."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        raise RuntimeError("csa_torch needs torch's headers")
    if not force and not binding_stale():
        return BINDING
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = BINDING + ".%d.tmp" % os.getpid()
    inc = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wno-deprecated-declarations",
           *["-I" + i for i in inc], BINDING_SRC, "-o", tmp, "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for csa_torch:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile libcsa.so, and csa_torch.so beside it where torch is, if missing or stale; returns libcsa's path."""
    pending = None
    if _torch_dir() is not None and (force or binding_stale()):
        pending = cf.ThreadPoolExecutor(max_workers=1).submit(build_binding, force)
    path = build_library(force, verbose, ptxas_info)
    if pending is not None:
        pending.result()
    return path


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile libcsa.so if missing or stale (all that importing the package needs); returns its path."""
    if not force and not stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    exe = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [exe, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
        return obj, res.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose or ptxas_info:
        for obj, err in results:
            if err:
                print(err)
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [exe, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))

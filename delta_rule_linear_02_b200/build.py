"""Build libefla.so (all CUDA sources of csrc/) in-tree for sm_100a with nvcc, and the binding's native part."""
from __future__ import annotations

import glob
import importlib.util
import os
import runpy
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libefla.so")
# the checked build: every direct global access and computed shared-memory store of the
# tensor-core forward is tested against its buffer (EFLA_CHECKED=1 in csrc/efla_common.cuh)
LIB_CHECKED = os.path.join(PKG, "libefla_checked.so")
# the binding's short way for small calls (csrc/efla_native.cpp), a Python extension module
LIB_NATIVE = os.path.join(PKG, "_efla_native.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _native_stale(mark: str, deps) -> bool:
    """Whether the binding's native part is missing, older than its sources, or built against another torch or Python."""
    if not os.path.exists(LIB_NATIVE) or os.path.getmtime(LIB_NATIVE) < max(map(os.path.getmtime, deps)):
        return True
    with open(LIB_NATIVE, "rb") as f:
        return f"efla native: {mark}\0".encode() not in f.read()


def build_native(force: bool = False, verbose: bool = False) -> str:
    source = os.path.join(CSRC, "efla_native.cpp")
    deps = [source, os.path.join(INCLUDE, "efla.h"), os.path.abspath(__file__)]
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    version = runpy.run_path(os.path.join(torch, "version.py"))["__version__"]
    mark = f"torch {version}, {sysconfig.get_config_var('SOABI')}"
    if not force and not _native_stale(mark, deps):
        return LIB_NATIVE
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = LIB_NATIVE + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-DNDEBUG", "-I", INCLUDE,
           f'-DEFLA_BUILT_FOR="{mark}"', f'-DEFLA_TORCH_VERSION="{version}"',
           *(f"-I{d}" for d in (os.path.join(torch, "include"), os.path.join(torch, "include/torch/csrc/api/include"),
                                sysconfig.get_paths()["include"], os.path.join(cuda, "include"))),
           "-o", tmp, source, f"-L{os.path.join(torch, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_NATIVE)
    return LIB_NATIVE


def build(force: bool = False, verbose: bool = False, extra=(), checked: bool = False) -> str:
    out = LIB_CHECKED if checked else LIB
    if not checked:
        build_native(force=force, verbose=verbose)
    if not force and not _stale(out):
        return out
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = out + f".tmp{os.getpid()}"
    flags = list(extra) + (["-DEFLA_CHECKED=1"] if checked else [])
    cmd = [nvcc, *NVCC_FLAGS, *flags, "-I", INCLUDE, "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, checked="--checked" in sys.argv))

"""Build libgdn.so in-tree with nvcc for sm_100a, and the compiled torch binding.

    python -m gated_deltanet_linear_chunked_b200.build [--force]

Compiles every ``csrc/*.cu`` into one shared library beside this file
(``libgdn.so``), exporting the C ABI declared in ``include/gdn.h``.  The CUDA
runtime is linked statically, so the library loads on a machine without a
GPU (the ABI tests use that); the CUDA driver API (tensor maps) is reached at run
time through ``cudaGetDriverEntryPoint``.

``csrc/torch_bind.cpp``, the argument marshalling of the softmax blocks'
operators, becomes ``_gdn_torch.so`` with g++ against the installed torch; it does
not link libgdn.so (the loader hands it the entry points' addresses).
"""
from __future__ import annotations

import glob
import hashlib
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libgdn.so")
BIND_SRC = os.path.join(CSRC, "torch_bind.cpp")
BIND_PATH = os.path.join(PKG, "_gdn_torch.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-Xptxas", "-warn-spills",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "gdn.h")]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libgdn.so if it is missing or older than its sources."""
    if not force and not is_stale():
        return LIB_PATH
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB_PATH + ".tmp.%d" % os.getpid()
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-shared", "-o", tmp,
           *sources(), "-lpthread"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True, cwd=PKG)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _bind_tag() -> str:
    """What the binding's compiled code depends on besides its own sources: torch's C++
    layout and internal entries, and the interpreter's ABI."""
    import sysconfig

    import torch
    return "torch %s, git %s, cxx11 abi %d, python %s" % (
        torch.__version__, torch.version.git_version, int(torch.compiled_with_cxx11_abi()),
        sysconfig.get_config_var("SOABI"))


def _bind_stamp(path: str) -> str:
    """The tag and the digest of the binding at `path`, as kept beside it."""
    with open(path, "rb") as f:
        return "%s\n%s\n" % (_bind_tag(), hashlib.sha256(f.read()).hexdigest())


def bind_is_stale() -> bool:
    """Missing, older than its sources, or built against another torch or Python."""
    if not os.path.exists(BIND_PATH):
        return True
    t = os.path.getmtime(BIND_PATH)
    if any(os.path.getmtime(p) > t for p in (BIND_SRC, os.path.join(INCLUDE, "gdn.h"))):
        return True
    try:
        with open(BIND_PATH + ".stamp") as f:
            return f.read() != _bind_stamp(BIND_PATH)
    except OSError:
        return True


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """Compile _gdn_torch.so if it is missing or stale."""
    if not force and not bind_is_stale():
        return BIND_PATH
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    tmp = BIND_PATH + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-DTORCH_EXTENSION_NAME=_gdn_torch",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
           "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], BIND_SRC, "-o", tmp,
           "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True, cwd=PKG)
    stamp = _bind_stamp(tmp)
    with open(tmp + ".stamp", "w") as f:
        f.write(stamp)
    os.replace(tmp, BIND_PATH)  # until the stamp follows, the binding counts as stale
    os.replace(tmp + ".stamp", BIND_PATH + ".stamp")
    return BIND_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    build_bind(force="--force" in sys.argv, verbose=True)

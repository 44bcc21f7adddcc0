"""Builds the sm_100a CUDA library ``libress.so`` in-tree with nvcc, and the
binding's C++ part ``_ress_call.so`` with the host compiler.

    python -m block_sparse_global_mean_b200.build
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libress.so")
CALL_PATH = os.path.join(PKG_DIR, "_ress_call.so")
CALL_TAG_PATH = CALL_PATH + ".tag"   # what call_tag() was when it was built
CALL_SOURCE = os.path.join(CSRC, "ress_call.cpp")
HEADER = os.path.join(PKG_DIR, "..", "include", "ress.h")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
    "--expt-relaxed-constexpr",
    "-shared",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(path: str, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def needs_build() -> bool:
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return _older(LIB_PATH, deps + [HEADER])


def call_tag() -> str:
    """The torch and Python whose object layouts the binding's C++ part holds."""
    import torch
    return (f"torch {torch.__version__} {getattr(torch.version, 'git_version', '')} "
            f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('SOABI')}")


def _call_current(tag: str) -> bool:
    try:
        with open(CALL_TAG_PATH) as f:
            return f.read() == tag and not _older(CALL_PATH, [CALL_SOURCE, HEADER])
    except OSError:
        return False


def build_call(force: bool = False, verbose: bool = False) -> str:
    """Compile the binding's C++ part against the installed torch; returns its path."""
    import torch
    tag = call_tag()
    if not force and _call_current(tag):
        return CALL_PATH
    for path in (CALL_TAG_PATH, CALL_PATH):   # one that does not fit is not left behind
        if os.path.exists(path):
            os.remove(path)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = CALL_PATH + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DRESS_CALL_TAG="{tag}"',
           *(f"-I{d}" for d in (os.path.join(root, "include"), os.path.join(cuda, "include"),
                                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"])),
           "-o", tmp, CALL_SOURCE, f"-L{os.path.join(root, 'lib')}",
           "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALL_PATH)
    with open(CALL_TAG_PATH, "w") as f:
        f.write(tag)
    return CALL_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every .cu under csrc/ into libress.so (sm_100a); returns its path.  The
    binding's C++ part is built behind it where torch's and Python's headers and a
    host compiler allow: without it the same calls are made through ctypes."""
    if force or needs_build():
        tmp = LIB_PATH + ".tmp"
        cmd = [_nvcc(), *NVCC_FLAGS, *extra_flags, "-o", tmp, *sources()]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB_PATH)
    try:
        build_call(force, verbose)
    except (ImportError, OSError, RuntimeError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the binding's C++ part was not built, its calls go through ctypes: {e}",
                      RuntimeWarning, stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])

"""In-tree build of the CUDA library (libcsa2.so) for sm_100a with nvcc, which needs nothing else, and, where torch
is installed, of the module with the Python calls of the paged key/value operators with g++ against its headers."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libcsa2.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "csa2.h")]
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in deps)


def bind_path() -> str:
    """The module with the Python calls: it serves the torch and the Python that it was built with."""
    import torch
    return os.path.join(PKG, f"_bind.{torch.__version__}.{sys.implementation.cache_tag}.so")


def _build_bind(force: bool) -> None:
    src, header, out = os.path.join(CSRC, "bind.cpp"), os.path.join(ROOT, "include", "csa2.h"), bind_path()
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    libs = os.path.join(home, "lib")
    dirs = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(home, "include"),
            os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                           *[f"-I{d}" for d in dirs], src, "-o", out, f"-L{libs}", f"-Wl,-rpath,{libs}",
                           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale():
        cmd = ["nvcc", *ARCH, *FLAGS, *sources(), "-o", LIB]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.check_call(cmd)
    try:
        import torch  # noqa: F401
    except ImportError:  # the C ABI alone
        return LIB
    _build_bind(force)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

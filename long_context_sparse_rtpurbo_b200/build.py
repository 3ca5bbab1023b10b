"""Builds librtp.so (sm_100a) in-tree with nvcc, and the native Python binding of its paged calls
(_binding.so) with g++."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-shared", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def cuda_include() -> str:
    """The headers of the toolkit that nvcc belongs to."""
    exe = shutil.which(nvcc())
    home = os.path.dirname(os.path.dirname(os.path.realpath(exe))) if exe else "/usr/local/cuda"
    for inc in (os.path.join(home, "include"), os.path.join(home, "targets", "x86_64-linux", "include"),
                "/usr/local/cuda/include"):
        if os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
            return inc
    raise RuntimeError(f"cuda_runtime_api.h not found beside {exe or 'nvcc'}")


def build(verbose: bool = False, extra_flags=(), out_name: str = "librtp.so") -> str:
    """Compiles csrc/rtp_api.cu into ``out_name`` (librtp_trace.so with -DRTP_TRACE records
    per-CTA phase timestamps of the decode kernel in the workspace)."""
    out = os.path.join(HERE, out_name)
    src = os.path.join(HERE, "csrc", "rtp_api.cu")
    cmd = [nvcc(), *NVCC_FLAGS, *extra_flags, "-o", out, src]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    return out


def build_checks(verbose: bool = False) -> str:
    """librtp_checks.so: the library with -DRTP_CHECKS (bounds checks of data-dependent indices
    that record RTP_ECHECK instead of touching memory outside a buffer), for debugging runs
    selected with RTP_LIBRARY_PATH."""
    return build(verbose, ["-DRTP_CHECKS"], "librtp_checks.so")


def build_binding(verbose: bool = False) -> str:
    """_binding.so: Python calls of the paged entry points (csrc/binding.cpp). It calls librtp.so by
    address and links only against the PyTorch that is installed."""
    import torch
    from torch.utils import cpp_extension as ext
    out = os.path.join(HERE, "_binding.so")
    inc = [sysconfig.get_paths()["include"], cuda_include(), *ext.include_paths()]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{d}" for d in inc], os.path.join(HERE, "csrc", "binding.cpp"), "-o", out,
           f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    return out


if __name__ == "__main__":
    print(build_binding(verbose=True))
    print(build(verbose=True))

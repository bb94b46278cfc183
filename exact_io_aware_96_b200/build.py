"""Build libfa.so (the CUDA library) in-tree with nvcc for sm_100a, and
_fa_torch.so (the torch side of differential attention and rotary positions,
host code only) with the C++ compiler against the installed torch. libfa.so
alone needs neither torch nor Python's headers: without them _fa_torch.so is
left out, with a note on stderr.

Usage: ``python -m exact_io_aware_96_b200.build`` (or ``__graft_entry__.build()``).
The CUDA runtime is linked statically; the driver API is reached through
cudaGetDriverEntryPoint, so the library needs no libcuda at link time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfa.so")
SOURCES = [os.path.join(CSRC, "fa_api.cu")]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


LIB_CHECK = os.path.join(HERE, "libfa_check.so")


TORCH_SOURCE = os.path.join(CSRC, "fa_torch.cpp")
TORCH_LIB = os.path.join(HERE, "_fa_torch.so")


def torch_missing() -> str | None:
    """What _fa_torch.so cannot be built without and is not here, or None."""
    import sysconfig
    try:
        import torch
    except ImportError:
        return "torch"
    for header in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                   os.path.join(os.path.dirname(torch.__file__), "include", "ATen", "ATen.h")):
        if not os.path.exists(header):
            return header
    return None


def build_torch() -> str:
    """Build _fa_torch.so, unless it is newer than its sources."""
    import sysconfig

    import torch
    sources = [TORCH_SOURCE, os.path.join(INCLUDE, "fa.h"), torch.__file__]
    if os.path.exists(TORCH_LIB) and all(os.path.getmtime(TORCH_LIB) > os.path.getmtime(s) for s in sources):
        return TORCH_LIB
    at = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [shutil.which("g++") or "g++", "-shared", "-fPIC", "-O2", "-std=c++17",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *("-I" + d for d in (INCLUDE, os.path.join(at, "include"),
                                os.path.join(at, "include", "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"], cuda)),
           "-o", TORCH_LIB + ".tmp", TORCH_SOURCE, "-L" + os.path.join(at, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("the C++ compiler failed:\n" + res.stdout + res.stderr)
    os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    return TORCH_LIB


def build(verbose: bool = False, extra: list[str] | None = None, check: bool = False) -> str:
    """Build libfa.so (and _fa_torch.so), or with check=True libfa_check.so: the
    same sources compiled with FA_CHECK=1 (device-side index and bounds checks)."""
    out = LIB_CHECK if check else LIB
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-shared",
           "-I" + INCLUDE, "-I" + CSRC, "-o", out + ".tmp", *(["-DFA_CHECK=1"] if check else []), *SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    if extra:
        cmd[1:1] = extra
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    os.replace(out + ".tmp", out)
    if verbose:
        sys.stdout.write(res.stdout + res.stderr)
    if not check:
        if missing := torch_missing():
            print(f"_fa_torch.so is not built (differential attention and rotary positions from Python need it): "
                  f"{missing} is missing", file=sys.stderr)
        else:
            build_torch()
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, check="--check" in sys.argv))

"""Build libsa.so in-tree with nvcc for sm_100a, and the binding's _fastcall.so.

    python -m sparse_attention_aware_b200.build [--force] [--ptxas-verbose]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsa.so")
FAST = os.path.join(PKG, "_fastcall.so")
FAST_SRC = os.path.join(CSRC, "fastcall.cpp")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def nvcc() -> str:
    for cand in [os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"]:
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _made_for() -> str:
    """What the native calls are compiled against, as they carry it."""
    import torch
    return "sa-fastcall for torch %s, python %d.%d;" % (torch.__version__, *sys.version_info[:2])


def fastcall_fits() -> bool:
    """Whether there are native calls, and compiled against this torch and Python."""
    try:
        with open(FAST, "rb") as f:
            return _made_for().encode() in f.read()
    except OSError:
        return False


def _fastcall_fresh() -> bool:
    deps = [FAST_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return fastcall_fits() and all(os.path.getmtime(p) <= os.path.getmtime(FAST) for p in deps)


def build_fastcall(force: bool = False) -> str:
    """The short calls of the binding, a Python module against torch's own
    libraries (already loaded by whoever imports it)."""
    if not force and _fastcall_fresh():
        return FAST
    import torch
    base = os.path.dirname(torch.__file__)
    tmp = FAST + ".tmp.%d" % os.getpid()
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
                    "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
                    '-DSA_MADE_FOR="%s"' % _made_for(), "-I", INCLUDE, "-isystem", os.path.join(base, "include"),
                    "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                    "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
                    FAST_SRC, "-o", tmp, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cuda",
                    "-ltorch_cpu", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, FAST)
    return FAST


def _try_fastcall(force: bool) -> None:
    """The binding does without its native calls (in Python, 8 to 20 us a call more)
    where they cannot be built; ones that are out of date are not left behind."""
    try:
        build_fastcall(force)
    except Exception as e:   # no compiler, headers or torch libraries, or not fitting ones
        if os.path.exists(FAST) and not _fastcall_fresh():
            os.remove(FAST)
        warnings.warn("the binding's native calls were not built: %s" % e, RuntimeWarning)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or _stale():
        _build_lib(verbose_ptxas)
    _try_fastcall(force)
    return LIB


def _build_lib(verbose_ptxas: bool) -> None:
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
           "-I", INCLUDE, "-I", CSRC, "-DSA_BUILD", *sources(), "-o", tmp]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="--ptxas-verbose" in sys.argv)
    print(LIB)

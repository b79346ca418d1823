"""Build libsplitzip.so in-tree with nvcc for sm_100a (B200), and the compiled
part of the Python binding (_binding.so) with g++ against torch's headers."""
from __future__ import annotations

import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
LIB_PATH = os.path.join(PKG, "libsplitzip.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "sz_binding.cpp")

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "splitzip.h")]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _deps())


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu into libsplitzip.so (skipped when up to date)."""
    if not force and not is_stale():
        return LIB_PATH
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [nvcc()] + NVCC_FLAGS + ["-I" + INCLUDE, "-o", tmp] + _sources()
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.check_call(cmd)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def binding_made_for() -> str:
    """What a compiled binding fits: it reads torch's and Python's structures."""
    import sysconfig

    import torch
    return "made for torch %s, python %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def binding_is_stale() -> bool:
    if not os.path.exists(BINDING_PATH):
        return True
    t = os.path.getmtime(BINDING_PATH)
    if any(os.path.getmtime(p) > t for p in (BINDING_SOURCE, os.path.join(INCLUDE, "splitzip.h"))):
        return True
    with open(BINDING_PATH, "rb") as f:
        return binding_made_for().encode() + b"\0" not in f.read()


def build_binding(force: bool = False) -> str:
    """Compile csrc/sz_binding.cpp into _binding.so (skipped when up to date)."""
    if not force and not binding_is_stale():
        return BINDING_PATH
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    dirs = include_paths() + [sysconfig.get_paths()["include"], INCLUDE, os.path.join(cuda, "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), '-DSZ_MADE_FOR="%s"' % binding_made_for()]
    cmd += ["-isystem" + d for d in dirs] + [BINDING_SOURCE, "-o", tmp, "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH

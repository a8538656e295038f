"""Builds libstreamkl.so in-tree with nvcc for sm_100a (no GPU needed).

    python -m attention_kl_divergence_02_b200.build [--force]
"""
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libstreamkl.so")
MAIN = os.path.join(CSRC, "streamkl.cu")
INCLUDE = os.path.join(ROOT, "include")
FASTCALL = os.path.join(PKG, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
FASTCALL_MAIN = os.path.join(CSRC, "fastcall.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    out = [os.path.join(INCLUDE, "streamkl.h")]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    return out


def stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build_fastcall(force=False):
    """Compile the CPython extension that shortens the paged calls, where Python's headers are installed (the
    binding does without it)."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return None
    made_of = (FASTCALL_MAIN, os.path.join(INCLUDE, "streamkl.h"))
    if not force and os.path.exists(FASTCALL) and all(os.path.getmtime(s) <= os.path.getmtime(FASTCALL) for s in made_of):
        return FASTCALL
    import torch
    at = os.path.dirname(torch.__file__)
    lib = os.path.join(at, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    tmp = FASTCALL + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()), "-I", INCLUDE, "-I", include]
    for path in (os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"), cuda):
        cmd += ["-isystem", path]
    cmd += ["-o", tmp, FASTCALL_MAIN, "-L", lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    subprocess.check_call(cmd)
    os.replace(tmp, FASTCALL)
    return FASTCALL


def build(force=False, verbose=False):
    """Compile the library if any source is newer than it, and the binding's extension.  Returns the library's path."""
    build_fastcall(force)
    if not force and not stale():
        return LIB
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [_nvcc()] + NVCC_FLAGS + ["-I", INCLUDE, "-I", CSRC, "-o", tmp, MAIN]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

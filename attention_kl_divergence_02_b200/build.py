"""Builds libstreamkl.so in-tree with nvcc for sm_100a (no GPU needed).

    python -m attention_kl_divergence_02_b200.build [--force]
"""
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libstreamkl.so")
MAIN = os.path.join(CSRC, "streamkl.cu")
INCLUDE = os.path.join(ROOT, "include")
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


def fastcall_path(torch_version):
    """Where the extension for a torch version lies: it calls torch's C++ interface, so one that was compiled with
    another version's headers is not to be loaded."""
    return os.path.join(PKG, "_fastcall-torch" + torch_version + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def build_fastcall(force=False):
    """Compile the CPython extension that shortens the paged calls, where Python's headers are installed (the
    binding does without it).  Returns its path or None."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return None
    import torch
    path = fastcall_path(torch.__version__)
    made_of = (FASTCALL_MAIN, os.path.join(INCLUDE, "streamkl.h"))
    if not force and os.path.exists(path) and all(os.path.getmtime(s) <= os.path.getmtime(path) for s in made_of):
        return path
    at = os.path.dirname(torch.__file__)
    lib = os.path.join(at, "lib")
    nvcc = os.path.realpath(shutil.which(_nvcc()) or _nvcc())
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    tmp = path + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()), "-I", INCLUDE, "-I", include]
    for header in (os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"), cuda):
        cmd += ["-isystem", header]
    cmd += ["-o", tmp, FASTCALL_MAIN, "-L", lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    subprocess.check_call(cmd)
    os.replace(tmp, path)
    return path


def build_library(force=False, verbose=False):
    """Compile the library if any source is newer than it."""
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


def build(force=False, verbose=False):
    """The library, which needs nvcc alone, and then the binding's extension, whose failure is a warning.  Returns
    the library's path."""
    build_library(force, verbose)
    try:
        build_fastcall(force)
    except Exception as e:      # no torch, a CPU-only one, no g++, headers that do not fit
        warnings.warn("the extension that shortens the paged calls was not built (%s: %s); they work without it"
                      % (type(e).__name__, e))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

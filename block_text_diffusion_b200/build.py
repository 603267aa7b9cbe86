"""Compile the CUDA library (libdg.so) and the serving binding (_serving.so)
in-tree, for sm_100a.

The shared object is written next to this file; `python -m
block_text_diffusion_b200.build` rebuilds it when any source is newer.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libdg.so")
SOURCES = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu*")) + glob.glob(os.path.join(HERE, "csrc", "*.inc"))) + sorted(glob.glob(os.path.join(ROOT, "include", "*.h")))
UNITS = ("dg_engine.cu", "dg_noalloc.cu", "dg_serve.cu")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


# The Python side of the serving operators: C++ against torch's headers.  Beside
# it stands what it was compiled for: another torch or Python needs another one.
BINDING = os.path.join(HERE, "_serving.so")
BINDING_KEY = os.path.join(HERE, "_serving.key")
BINDING_SOURCES = [os.path.join(HERE, "csrc", "dg_serving_py.cpp"), os.path.join(ROOT, "include", "dg.h")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in SOURCES)


def binding_key() -> str:
    """What a compiled binding depends on besides its sources."""
    import torch
    return f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sys.version.split()[0]}\n"


def binding_built_for() -> str:
    """The binding_key of the binding that is there ("" if unknown)."""
    if not os.path.exists(BINDING_KEY):
        return ""
    with open(BINDING_KEY) as f:
        return f.read()


def _binding_paths():
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(cuda, "include")], os.path.join(root, "lib")


def binding_lacks() -> str:
    """Why the binding cannot be compiled here ("": it can).  libdg.so needs nvcc alone."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return "torch is not installed"
    if shutil.which("g++") is None:
        return "g++ is not installed"
    try:
        dirs, lib = _binding_paths()
    except RuntimeError as e:
        return str(e)
    for f in ("c10/cuda/CUDAStream.h", "torch/csrc/autograd/python_variable.h", "Python.h", "cuda_runtime_api.h"):
        if not any(os.path.exists(os.path.join(d, f)) for d in dirs):
            return f"the header {f} is not installed"
    return "" if os.path.exists(os.path.join(lib, "libc10_cuda.so")) else "torch has no CUDA library"


def binding_fresh() -> bool:
    """The binding is there, newer than its sources, and for this torch and Python."""
    try:
        key = binding_key()
    except ImportError:
        return False
    return os.path.exists(BINDING) and binding_built_for() == key and all(
        os.path.getmtime(s) <= os.path.getmtime(BINDING) for s in BINDING_SOURCES)


def build_binding(force: bool = False) -> str:
    if not force and binding_fresh():
        return BINDING
    import torch
    dirs, lib = _binding_paths()
    tmp = BINDING + ".tmp%d" % os.getpid()
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
                           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                           *["-I" + d for d in dirs], "-o", tmp, BINDING_SOURCES[0], "-L" + lib,
                           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    os.replace(tmp, BINDING)
    with open(BINDING_KEY + ".tmp%d" % os.getpid(), "w") as f:
        f.write(binding_key())
    os.replace(f.name, BINDING_KEY)
    return BINDING


def build(force: bool = False, verbose: bool = False, lib: str = LIB) -> str:
    if force or lib != LIB or stale():
        tmp = lib + ".tmp%d" % os.getpid()
        cmd = [nvcc(), "-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "-shared",
               "-o", tmp, "--threads", "0", *(os.path.join(HERE, "csrc", f) for f in UNITS)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.check_call(cmd)
        os.replace(tmp, lib)
    if lib == LIB and (force or not binding_fresh()):
        lacks = binding_lacks()
        if lacks:
            print(f"the Python side of the serving operators is not built: {lacks}", file=sys.stderr)
        else:
            build_binding(force=True)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

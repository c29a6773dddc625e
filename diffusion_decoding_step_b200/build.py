"""Build libdllm.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and the
torch binding of its paged cache calls with the host compiler."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdllm.so")
# The same sources with DLLM_DEBUG: row positions read from device memory are
# range-checked in the kernels (an error bit instead of an access).
LIB_DEBUG = os.path.join(HERE, "libdllm_debug.so")
SOURCES = ["api.cu", "gemm.cu", "attn.cu", "small.cu", "stack.cu", "paged_api.cu", "paged.cu"]
# Python module that takes torch tensors (csrc/paged_torch.cpp)
BINDING = os.path.join(HERE, "_paged_torch.so")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    deps.append(os.path.join(HERE, "..", "include", "dllm.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build_binding(force: bool = False) -> str | None:
    """Compile the torch binding of the paged cache calls into _paged_torch.so; rebuilt
    when its sources, torch or Python are others than it was built with.  Without torch or
    Python's headers there is none: says so and returns None."""
    import sysconfig

    src = os.path.join(CSRC, "paged_torch.cpp")
    include = sysconfig.get_paths()["include"]
    try:
        import torch
    except ImportError as e:
        print(f"build: no torch ({e}): {os.path.basename(BINDING)} is left out", file=sys.stderr)
        return None
    if not os.path.exists(os.path.join(include, "Python.h")):
        print(f"build: no Python.h in {include}: {os.path.basename(BINDING)} is left out",
              file=sys.stderr)
        return None
    made_for = f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"
    stamp = BINDING + ".made_for"
    deps = [src, os.path.join(HERE, "..", "include", "dllm.h")]
    if not force and os.path.exists(BINDING) and os.path.exists(stamp) \
            and open(stamp).read() == made_for \
            and all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps):
        return BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + ".tmp"
    subprocess.run(
        [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I" + include, "-I" + os.path.join(root, "include"),
         "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
         "-I" + os.path.join(cuda, "include"), src, "-o", tmp,
         "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
         "-lc10_cuda"], check=True)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(made_for)
    return BINDING


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile every CUDA source into libdllm.so next to this file (with
    debug=True: libdllm_debug.so, the DLLM_DEBUG build), then the torch binding."""
    lib = LIB_DEBUG if debug else LIB
    if force or stale(lib):
        cmd = [nvcc(), *FLAGS]
        if debug:
            cmd += ["-DDLLM_DEBUG"]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        cmd += [os.path.join(CSRC, f) for f in SOURCES]
        tmp = lib + ".tmp"
        cmd += ["-o", tmp]
        subprocess.run(cmd, check=True)
        os.replace(tmp, lib)
    if not debug:
        build_binding(force)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                debug="--debug" in sys.argv))

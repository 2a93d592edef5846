"""Builds in-tree the CUDA library ``libpivot.so`` for sm_100a with nvcc, and the compiled half of the Python binding
(``_step``, host code alone, against the torch that is installed) with the host compiler.

    python -m query_group_top_b200.build [-v] [--library]      # --library: libpivot.so alone, which needs nvcc and no torch
"""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpivot.so")
BINDING = os.path.join(HERE, "_step" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILT_FOR = os.path.join(HERE, "_build", "step_built_for.txt")
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2", "-shared",
]


def sources():
    return sorted(os.path.join(SRC, f) for f in os.listdir(SRC) if f.endswith((".cu", ".cuh")))


def torch_version() -> str:
    """The installed torch's version, without importing it."""
    from importlib.metadata import version
    return version("torch")


def built_for():
    """The torch that the binding was compiled against, None if that is not known."""
    try:
        with open(BUILT_FOR) as f:
            return f.read().strip()
    except OSError:
        return None


def stale(target=LIB) -> bool:
    if not os.path.exists(target):
        return True
    if target == BINDING and built_for() != torch_version():
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(SRC, "binding.cpp")] if target == BINDING else sources()
    return any(os.path.getmtime(s) > t for s in [*deps, os.path.join(ROOT, "include", "pivot.h")])


def _run(cmd, target, verbose):
    tmp = target + f".tmp{os.getpid()}"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, target)


def build_binding(verbose: bool = False) -> str:
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DPIVOT_TORCH="{torch_version()}"', "-I", os.path.join(ROOT, "include"),
          "-isystem", os.path.join(at, "include"), "-isystem", os.path.join(at, "include", "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
          os.path.join(SRC, "binding.cpp"), "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python"], BINDING, verbose)
    os.makedirs(os.path.dirname(BUILT_FOR), exist_ok=True)
    with open(BUILT_FOR, "w") as f:
        f.write(torch_version() + "\n")
    return BINDING


def build(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    """The library, and with `binding` the compiled half of the binding, where they are missing or stale."""
    if force or stale(LIB):
        nvcc = os.environ.get("NVCC", "nvcc")
        _run([nvcc, *(["-Xptxas=-v"] if verbose else []), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"),
              os.path.join(SRC, "pivot.cu")], LIB, verbose)
    if binding and (force or stale(BINDING)):
        build_binding(verbose)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv, binding="--library" not in sys.argv)
    print(LIB)

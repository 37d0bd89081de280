"""Build step: compile libstepmoe.so in-tree for sm_100a (nvcc cross-compiles without a GPU)."""
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libstepmoe.so")
PYARGS = os.path.join(HERE, "_pyargs.so")
SOURCES = ["api.cu", "route.cu", "permute.cu", "expert_ffn.cu", "combine.cu", "pack.cu", "noalloc.cu", "diag.cu", "fp8.cu", "selftest.cu",
           "expert_train.cu", "backward.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-shared",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def build_pyargs(verbose: bool = False) -> str:
    """The binding's native argument check (csrc/pyargs.cpp, a CPython module against the installed torch)."""
    from torch.utils.cpp_extension import include_paths, library_paths
    libs = library_paths()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-o", PYARGS,
           os.path.join(CSRC, "pyargs.cpp"), f"-I{sysconfig.get_paths()['include']}", "-I/usr/local/cuda/include",
           *[f"-I{p}" for p in include_paths()], *[f"-L{p}" for p in libs], *[f"-Wl,-rpath,{p}" for p in libs],
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    return PYARGS


def build(verbose: bool = False, extra_flags=()) -> str:
    cmd = ["nvcc", *NVCC_FLAGS, *extra_flags, "-o", LIB, *[os.path.join(CSRC, s) for s in SOURCES]]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    build_pyargs(verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True)

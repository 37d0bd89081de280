"""Build step: compile libstepmoe.so in-tree for sm_100a (nvcc cross-compiles without a GPU)."""
import os
import shutil
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
    """The binding's native training calls (csrc/pyargs.cpp, a CPython module against the installed torch)."""
    from torch.utils import cpp_extension
    libs = cpp_extension.library_paths()
    cuda = cpp_extension.CUDA_HOME or os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-o", PYARGS,
           os.path.join(CSRC, "pyargs.cpp"), f"-I{sysconfig.get_paths()['include']}", f"-I{os.path.join(cuda, 'include')}",
           *[f"-I{p}" for p in cpp_extension.include_paths()], *[f"-L{p}" for p in libs], *[f"-Wl,-rpath,{p}" for p in libs],
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
    try:
        import torch  # noqa: F401
    except ImportError:   # the library needs no torch, and the binding makes its calls without the module
        print("torch is not installed: built the library alone")
    else:
        build_pyargs(verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True)

"""Build the CUDA library ``_build/liblynx.so`` for sm_100a, in-tree.

    python -m activation_sparse_gemm_lynx_b200.build [--force] [--verbose]

The host compiler also builds ``_build/_lynx_torch.<versions>.so`` from
``csrc/torch_binding.cpp``: the tensor marshalling of the calls that are short
on the device, linked to that library and to torch's own.  Its name holds the
Python ABI and the torch it was compiled against, so that another one's is never
loaded.  Where torch or the
Python headers are not there it is left out: users of ``include/lynx.h`` need nvcc
alone.

One nvcc invocation compiles every ``csrc/*.cu`` file with
``-gencode arch=compute_100a,code=sm_100a -lineinfo`` and links a shared
library with the CUDA runtime linked statically (the driver API is reached
through ``cudaGetDriverEntryPoint``), so the library loads on a machine
without a GPU driver and only needs one when a kernel is launched.
"""
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "liblynx.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-shared", "-cudart", "static", "--threads", "0",
]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                               glob.glob(os.path.join(CSRC, "*.h")) +
                               [os.path.join(INCLUDE, "lynx.h")])


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def binding_path() -> str:
    """Where the tensor marshalling for the running Python and torch is (or would be)."""
    import torch

    tag = "%s-torch%s-cxx11abi%d" % (sysconfig.get_config_var("SOABI"), torch.__version__,
                                     int(torch._C._GLIBCXX_USE_CXX11_ABI))
    return os.path.join(OUT_DIR, "_lynx_torch.%s.so" % re.sub(r"[^A-Za-z0-9.+-]", "_", tag))


def binding_up_to_date() -> bool:
    path = binding_path()
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t
               for f in (BINDING_SOURCE, os.path.join(INCLUDE, "lynx.h"), os.path.abspath(__file__)))


def binding_lacks() -> str:
    """What building the tensor marshalling would need and is not here ('' if nothing)."""
    if importlib.util.find_spec("torch") is None:
        return "torch is not installed"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "the Python headers are not installed"
    return ""


def build_binding() -> str:
    """Compile the tensor marshalling against torch; return its path."""
    import torch

    home = os.path.dirname(torch.__file__)
    path = binding_path()
    tmp = path + ".tmp%d" % os.getpid()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include")]
    cmd += ["-isystem", os.path.join(home, "include"),
            "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
            "-o", tmp, BINDING_SOURCE, "-L", OUT_DIR, "-llynx", "-Wl,-rpath,$ORIGIN",
            "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what any source is newer than; return the library's path."""
    if force or not up_to_date():
        build_library(verbose)
    lacks = binding_lacks()
    if lacks:
        print(f"tensor binding not built: {lacks}; {LIB} needs neither", file=sys.stderr)
    elif force or not binding_up_to_date():
        build_binding()
    return LIB


def build_library(verbose: bool = False) -> str:
    """Compile the CUDA library; return its path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *_sources()]
    if verbose:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))

"""Build librtp.so in-tree with nvcc for sm_100a (no torch involved), and the
Python binding of its paged calls, _paged.so, with g++ against torch.  _paged.torch
beside it names the Python and the torch it was built for; where those change it is
built again, where they or their headers are missing it is left out with a warning
(the paged calls then raise on first use).

    python -m long_context_sparse_rtp_b200.build [--force]
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "librtp.so")
BINDING = os.path.join(CSRC, "paged_binding.cpp")
EXT = os.path.join(HERE, "_paged.so")
STAMP = os.path.join(HERE, "_paged.torch")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-cudart", "static",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "rtp.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def binding_tag() -> str:
    """What a binding depends on beside its sources: this Python and this torch."""
    import torch
    return (f"python {sys.version_info.major}.{sys.version_info.minor} torch {torch.__version__} "
            f"cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}")


def binding_built_for() -> str:
    """The tag of the _paged.so that is there, empty without one."""
    if not (os.path.exists(EXT) and os.path.exists(STAMP)):
        return ""
    with open(STAMP) as f:
        return f.read().strip()


def binding_needs() -> list:
    """What is missing to build the binding."""
    if importlib.util.find_spec("torch") is None:
        return ["torch"]
    from torch.utils.cpp_extension import include_paths
    headers = {"Python.h": [sysconfig.get_paths()["include"]],
               "torch/csrc/autograd/python_variable.h": include_paths(device_type="cuda")}
    return [h for h, dirs in headers.items()
            if not any(os.path.exists(os.path.join(d, h)) for d in dirs)]


def build_binding(force: bool = False, verbose: bool = False) -> str:
    deps = [BINDING, os.path.join(INCLUDE, "rtp.h")]
    if not force and binding_built_for() == binding_tag() and \
            all(os.path.getmtime(d) <= os.path.getmtime(EXT) for d in deps):
        return EXT
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", sysconfig.get_paths()["include"]]
    for d in include_paths(device_type="cuda"):
        cmd += ["-isystem", d]
    cmd += ["-o", tmp, BINDING]
    for d in library_paths():
        cmd += ["-L", d]
    cmd += ["-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
            "-L", HERE, "-l:librtp.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, EXT)
    with open(tmp, "w") as f:
        f.write(binding_tag() + "\n")
    os.replace(tmp, STAMP)
    return EXT


def build(force: bool = False, verbose: bool = False) -> str:
    build_lib(force, verbose)
    missing = binding_needs()
    if missing:
        warnings.warn(f"the paged calls' binding is not built: no {' and no '.join(missing)}")
    else:
        build_binding(force, verbose)
    return LIB


def build_lib(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-shared", "-o", tmp, *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)

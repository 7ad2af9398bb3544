"""Build the in-tree shared library ``libtg_gemm.so`` for sm_100a with nvcc, and the
CPython module ``_calls.so`` that marshals torch tensors to its feed-forward calls.

Run ``python -m tiled_dense_gemm_fp16_b200.build`` (or call ``build()``).
Both are built in the package directory so that they travel with the source
tree; the library links cudart statically and looks the driver's tensor-map
encoder up at run time, so it needs no other CUDA library at load.  The module
links to torch and to the library beside it; without torch only the library is
built.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_PATH = os.path.join(HERE, "libtg_gemm.so")
CALLS_PATH = os.path.join(HERE, "_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")
SOURCES = [os.path.join(CSRC, "tg_gemm.cu")]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared",
              f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtg_gemm.so")


def _deps():
    deps = list(SOURCES)
    for name in os.listdir(CSRC):
        if name.endswith((".cuh", ".h")):
            deps.append(os.path.join(CSRC, name))
    deps.append(os.path.join(ROOT, "include", "tg_gemm.h"))
    return deps


def _older(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def is_stale() -> bool:
    return _older(LIB_PATH, _deps())


def calls_target() -> str:
    """What the compiled torch module is good for: it reads torch's objects by their layout and Python's by their ABI."""
    import sysconfig

    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sysconfig.get_config_var('SOABI')}")


def _calls_command(out: str) -> list[str]:
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda_dir = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    includes = [os.path.join(ROOT, "include"), os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda_dir, "include")]
    # nvcc's host compiler, not $CXX: one that links its own C++ runtime statically leaves two of them in the
    # process, and an exception that torch's code throws through the module ends it.
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in includes),
            CALLS_SOURCE, "-o", out, f"-L{HERE}", "-l:libtg_gemm.so", f"-L{os.path.join(torch_dir, 'lib')}", "-lc10",
            "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]


def _calls_key() -> str:
    """Target and build command of the module, which it carries as text."""
    import hashlib
    command = hashlib.sha256(" ".join(_calls_command("")).encode()).hexdigest()[:16]
    return f"{calls_target()}; built by {command}"


def calls_stale() -> bool:
    """Whether the module is missing, older than its sources, or built for another torch or Python or by another command."""
    if _older(CALLS_PATH, [CALLS_SOURCE, os.path.join(ROOT, "include", "tg_gemm.h")]):
        return True
    try:
        key = _calls_key() + "\0"
    except RuntimeError:  # no nvcc, so none to build it again with: what it was built for still counts
        key = calls_target() + "\0"
    with open(CALLS_PATH, "rb") as f:
        return key.encode() not in f.read()


def build_calls(force: bool = False, verbose: bool = False) -> str | None:
    """The torch module (None without torch).  Needs the library to link to."""
    import importlib.util
    if importlib.util.find_spec("torch") is None:
        return None
    if not force and not calls_stale():
        return CALLS_PATH
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = _calls_command(tmp)
    cmd += [f'-DTG_CALLS_TARGET="{calls_target()}"', f'-DTG_CALLS_KEY="{_calls_key()}"']
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALLS_PATH)
    return CALLS_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not is_stale():
        build_calls(False, verbose)
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, *SOURCES, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    build_calls(force, verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

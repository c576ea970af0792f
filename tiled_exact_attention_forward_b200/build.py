"""Build the CUDA library in-tree: csrc/*.cu -> libfa_b200.so (sm_100a only).

Run ``python -m tiled_exact_attention_forward_b200.build`` (or call
:func:`build`).  The compiler is nvcc from CUDA 12.9; nothing is JIT-compiled
at import time, and the built library sits next to this file so it travels
with the source tree.

Each source is compiled to an object of its own (in parallel) as whole-program
device code -- one module per source file, no device linking: under separate
compilation (-rdc) ptxas ignores the per-warpgroup register budgets that the
forward kernel sets with setmaxnreg -- then one nvcc call links them.  Flags can differ per file: the
float32 forward (the exact path of the single-head fp32 workload) and the
norm-and-rotate kernels (float32 in and out among their types) are built without
``--use_fast_math`` so their exp2, log, square root and division are the
IEEE-rounded ones; every other kernel calls its fast instructions explicitly and keeps the
fast-math flags it was measured with.

csrc/calls.cpp, the compiled side of some of the Python calls, becomes the extension
module _calls beside it (host code only, against torch's headers).  It serves the Python
and the torch that it was built for alone: its file name carries Python's tag, and it is
built again when built_for() is no longer what the last build noted.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libfa_b200.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
CALLS_SOURCE = os.path.join(CSRC, "calls.cpp")
CALLS_PATH = os.path.join(HERE, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON_FLAGS = [
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", os.path.join(ROOT, "include"),
]
FAST_MATH = ["--use_fast_math"]
# Sources built with IEEE-rounded float32 math (no --use_fast_math).
EXACT_MATH_SOURCES = {"fwd_f32.cu", "norm_rope.cu", "append_paged.cu"}


def nvcc() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA 12.9 toolkit is required to build the library")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def flags_for(src: str):
    """nvcc flags of one source file."""
    name = os.path.basename(src)
    return [*ARCH_FLAGS, *COMMON_FLAGS, *([] if name in EXACT_MATH_SOURCES else FAST_MATH)]


def _fresh(path, files) -> bool:
    """`path` is there and no older than this script, the C header or any of `files`."""
    files = [*files, *glob.glob(os.path.join(ROOT, "include", "*.h")), os.path.abspath(__file__)]
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def library_up_to_date() -> bool:
    headers = [f for pattern in ("*.cuh", "*.h") for f in glob.glob(os.path.join(CSRC, pattern))]
    return _fresh(LIB_PATH, sources() + headers)


def built_for() -> str:
    """The Python, torch and C++ ABI that the extension module is compiled against."""
    import torch

    return f"{sys.implementation.cache_tag} torch-{torch.__version__} abi-{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def _stamp() -> str:
    return os.path.join(OBJ_DIR, "calls.stamp")


def calls_up_to_date() -> bool:
    if not (_fresh(CALLS_PATH, [CALLS_SOURCE]) and os.path.exists(_stamp())):
        return False
    with open(_stamp()) as f:
        return f.read() == built_for()


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


def _compile(src: str, extra, verbose: bool):
    obj = os.path.join(OBJ_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *flags_for(src), *(extra or []), "-c", "-o", obj, src]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, cwd=CSRC, capture_output=True, text=True)
    return obj, r


def calls_command(out: str):
    """The host compiler's command for the extension module: the one torch was built to go with (a
    compiler that links a C++ runtime of its own would not share its exceptions)."""
    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    libs = ["torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda"]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DFA_BUILT_FOR="{built_for()}"',
            *(f"-I{d}" for d in inc), "-o", out, CALLS_SOURCE,
            *(f"-L{d}" for d in cpp_extension.library_paths()), *(f"-l{n}" for n in libs)]


def _build_calls(verbose: bool):
    tmp = CALLS_PATH + ".tmp"
    cmd = calls_command(tmp)
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, cwd=CSRC, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"the host compiler failed on calls.cpp with exit code {r.returncode} ({LIB_NAME} is built)")
    if os.path.exists(_stamp()):
        os.remove(_stamp())
    os.replace(tmp, CALLS_PATH)
    with open(_stamp(), "w") as f:
        f.write(built_for())


def _build_library(verbose: bool, extra_flags):
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, extra_flags, verbose), srcs))
    objs = []
    for (obj, r), src in zip(results, srcs):
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)} with exit code {r.returncode}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        objs.append(obj)
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, cwd=CSRC, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"nvcc link failed with exit code {r.returncode}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile every kernel for sm_100a into libfa_b200.so, and the extension module; returns the
    library's path.  What is up to date stays as it is."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    # Side by side; the library does not need the module, which a machine without Python's or
    # torch's headers cannot build.
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_build_calls, verbose) if force or not calls_up_to_date() else None
        if force or not library_up_to_date():
            _build_library(verbose, extra_flags)
    if calls is not None:
        calls.result()
    return LIB_PATH


if __name__ == "__main__":
    v = "-v" in sys.argv
    flags = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force="--force" in sys.argv, verbose=v or bool(flags), extra_flags=flags))

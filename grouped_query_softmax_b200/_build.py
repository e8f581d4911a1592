"""Build libgqa.so in-tree with nvcc for sm_100a, and _torch_calls.so, the torch side of the calls
around the paged cache, with g++ against the installed torch (no JIT cache, no pip install)."""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgqa.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCES = ["gqa_kernels.cu", "gqa_api.cpp", "gqa_decode_static.cu", "gqa_host.cpp", "gqa_cache.cu"]
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared", "-cudart", "static",
    "-I", os.path.join(ROOT, "include"),
]


CALLS = os.path.join(HERE, "_torch_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")


def _torch_dir():
    """The installed torch's folder, or None where _torch_calls.so cannot be built: no torch, or one
    without CUDA. libgqa.so and its C ABI need neither. torch itself is not imported."""
    spec = importlib.util.find_spec("torch")
    where = next(iter(spec.submodule_search_locations or ()), None) if spec else None
    return where if where and os.path.exists(os.path.join(where, "lib", "libc10_cuda.so")) else None


def _built_for(torch):
    """What _torch_calls.so is compiled against, written into it: torch's and Python's C++ interfaces
    change with their versions."""
    try:
        with open(os.path.join(torch, "version.py")) as f:
            version = re.search(r"__version__\s*=\s*['\"]([^'\"]+)", f.read()).group(1)
    except (OSError, AttributeError):
        version = "unknown"
    return "built for torch %s, %s" % (version, sysconfig.get_config_var("SOABI"))


def _calls_command(out):
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(NVCC))
    paths = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
             os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            '-DGQA_BUILT_FOR="%s"' % _built_for(torch), "-o", out, CALLS_SOURCE,
            *[x for d in paths for x in ("-isystem", d)], "-L" + os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]


def _calls_stale():
    torch = _torch_dir()
    if torch is None:
        return False  # nothing to build it with
    if not os.path.exists(CALLS):
        return True
    t = os.path.getmtime(CALLS)
    if any(os.path.getmtime(p) > t for p in (CALLS_SOURCE, os.path.join(ROOT, "include", "gqa.h"))):
        return True
    with open(CALLS, "rb") as f:
        return _built_for(torch).encode() + b"\0" not in f.read()


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(ROOT, "include", "*.h")))


def stale() -> bool:
    return _lib_stale() or _calls_stale()


def _lib_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile the CUDA library and, where torch is installed, the torch side; returns the library's
    path. Raises CalledProcessError on failure."""
    for path, old, command in (
            (LIB, _lib_stale, lambda tmp: [NVCC, *FLAGS, *extra_flags, "-o", tmp, *[os.path.join(CSRC, s) for s in SOURCES]]),
            (CALLS, _calls_stale, _calls_command)):
        if path == CALLS and _torch_dir() is None:
            print("_torch_calls.so is not built: no torch with CUDA is installed. The C ABI does without.")
            continue
        if not force and not old():
            continue
        tmp = path + ".tmp%d" % os.getpid()
        cmd = command(tmp)
        if verbose:
            print(" ".join(cmd))
        subprocess.check_call(cmd)
        os.replace(tmp, path)
    return LIB


if __name__ == "__main__":
    import sys
    build(force=True, verbose=True, extra_flags=sys.argv[1:])

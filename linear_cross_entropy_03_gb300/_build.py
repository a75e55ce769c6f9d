"""Builds the CUDA library in-tree: csrc/*.cu -> _lib/libflce03.so (sm_103a), and
the Python extension that calls it with tensors: csrc/binding.cpp ->
_lib/flce_torch-<torch version>.so.

Each translation unit is compiled by its own process (in parallel), then linked,
the library with the static CUDA runtime.  A rebuild happens only when a source
or header is newer than what is built.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB = os.path.join(OUT_DIR, "libflce03.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def binding_path() -> str:
    import torch
    return os.path.join(OUT_DIR, f"flce_torch-{torch.__version__}.so")


def binding_obstacle():
    """Why the extension cannot be built here (the library needs none of it), or None."""
    if importlib.util.find_spec("torch") is None:
        return "torch is not installed"
    header = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return None if os.path.exists(header) else f"{header} is missing"


def _inputs():
    return _sources() + [os.path.join(CSRC, "binding.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "flce.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    built = [LIB] if binding_obstacle() else [LIB, binding_path()]
    if not all(map(os.path.exists, built)):
        return False
    t = min(map(os.path.getmtime, built))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _run(what: str, cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_binding(nvcc: str):
    """The extension's object file, and the command that links it once the library is there."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cxx, obj = os.environ.get("CXX", "g++"), os.path.join(OUT_DIR, "binding.o")
    _run(f"{cxx} on binding.cpp", [
        cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in include),
        "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    return [cxx, "-shared", obj, LIB, f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Builds what is not up to date and returns the library's path.

    Where the extension cannot be built the library is built all the same; the
    functions that take tensors then raise when they are called.
    """
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    objs = [os.path.join(OUT_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]
    obstacle = binding_obstacle()

    def compile_one(src, obj):
        return _run(f"nvcc on {os.path.basename(src)}", [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj])

    with concurrent.futures.ThreadPoolExecutor(len(srcs) + 1) as ex:
        binding = None if obstacle else ex.submit(_compile_binding, nvcc)
        logs = list(ex.map(compile_one, srcs, objs))
    if verbose:
        for s, log in zip(srcs, logs):
            if log.strip():
                print(f"--- {os.path.basename(s)}\n{log}")
    tmp = LIB + ".tmp"
    _run("link", [nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libflce03.so", "-o", tmp, *objs, "-lcudart_static",
                  "-ldl", "-lpthread", "-lrt"])
    os.replace(tmp, LIB)
    if binding is None:
        warnings.warn(f"only the library is built, and not the extension that calls it with tensors: {obstacle}")
        return LIB
    tmp = binding_path() + ".tmp"
    _run("link", [*binding.result(), "-o", tmp])
    os.replace(tmp, binding_path())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))

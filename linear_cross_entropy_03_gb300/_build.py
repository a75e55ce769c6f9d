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
import os
import shutil
import subprocess
import sysconfig

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


def _inputs():
    return _sources() + [os.path.join(CSRC, "binding.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "flce.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    built = (LIB, binding_path())
    if not all(map(os.path.exists, built)):
        return False
    t = min(map(os.path.getmtime, built))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    objs = [os.path.join(OUT_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src, obj):
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return r.stdout + r.stderr

    def compile_binding():
        import torch
        root = os.path.dirname(os.path.abspath(torch.__file__))
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
        include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        obj = os.path.join(OUT_DIR, "binding.o")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               *(f"-I{p}" for p in include), "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
        return obj, os.path.join(root, "lib")

    with concurrent.futures.ThreadPoolExecutor(len(srcs) + 1) as ex:
        binding = ex.submit(compile_binding)
        logs = list(ex.map(compile_one, srcs, objs))
    if verbose:
        for s, log in zip(srcs, logs):
            if log.strip():
                print(f"--- {os.path.basename(s)}\n{log}")
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libflce03.so", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    obj, torch_lib = binding.result()
    tmp = binding_path() + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB, f"-L{torch_lib}", "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, binding_path())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))

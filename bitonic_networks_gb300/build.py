"""Builds libgsort.so in-tree with nvcc for sm_103a (GB300), and the Python
module _ops (its language-model operators on torch tensors) with g++.

Each source compiles to an object in parallel; the CUDA objects link into one
shared library with the CUDA runtime linked statically, and _ops.so links
against it.  The library needs nvcc alone: where torch or g++ is missing it is
there all the same, and only _ops fails.  A build is skipped when its result is
newer than every source and header, and _ops is for the Python and the torch
that are installed.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libgsort.so")
OPS_PATH = os.path.join(PKG, "_ops.so")
OPS_STAMP = os.path.join(BUILD_DIR, "ops.stamp")     # what _ops.so was built for
BINDING = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libgsort")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer_than(path: str, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def library_up_to_date() -> bool:
    return _newer_than(LIB_PATH, sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
                       + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__])


def ops_match() -> bool:
    """Whether _ops.so is there and for this Python and this torch."""
    if not (os.path.exists(OPS_PATH) and os.path.exists(OPS_STAMP)):
        return False
    try:
        want = _ops_stamp()
    except RuntimeError:      # no torch
        return False
    with open(OPS_STAMP) as f:
        return f.read() == want


def up_to_date() -> bool:
    return (library_up_to_date() and ops_match()
            and _newer_than(OPS_PATH, [BINDING, __file__] + glob.glob(os.path.join(INCLUDE, "*.h"))))


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch is not installed: _ops, the language-model operators on torch tensors, needs it")
    return spec.submodule_search_locations[0]


def _ops_stamp() -> str:
    """The C++ module holds for one interpreter and one build of torch (its
    version file names both the version and the sources' commit)."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{f.read()}"


def _compile_binding() -> str:
    obj = os.path.join(BUILD_DIR, "binding.o")
    include = os.path.join(_torch_dir(), "include")
    dirs = [include, os.path.join(include, "torch", "csrc", "api", "include"),
            os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
            sysconfig.get_paths()["include"], INCLUDE]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", *[f for d in dirs for f in ("-isystem", d)], "-c", BINDING, "-o", obj],
         "g++ on binding.cpp")
    return obj


def _link_binding(obj: str):
    tmp = OPS_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu",
          "-lc10", "-lc10_cuda", "-L", PKG, "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN"], "link of _ops.so")
    os.replace(tmp, OPS_PATH)
    with open(OPS_STAMP, "w") as f:
        f.write(_ops_stamp())


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile the CUDA sources and link libgsort.so; returns its path."""
    if not force and not extra_flags and library_up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = _run(cmd, f"nvcc on {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(16, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-o", tmp, *objs], "link of libgsort.so")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build libgsort.so and _ops.so; returns the library's path.  The library
    is linked whatever becomes of _ops."""
    if not force and not extra_flags and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding)
        build_library(force, verbose, extra_flags)
        _link_binding(binding.result())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))

"""Builds the sm_100a shared library ``libfa_sm100.so`` in this directory.

Usage: ``python -m exact_tiled_attention_40_b200.build`` (or ``build()`` from
Python).  Every .cu file under csrc/ is compiled with nvcc for sm_100a only and
linked with the static CUDA runtime; the driver API is reached at run time
through cudaGetDriverEntryPoint, so loading the library needs no GPU.  The
compiled part of the Python binding, ``_step.so``, is built with g++ beside it,
where g++ and the headers of torch and Python are: the library needs neither.

``build(debug=True)`` (``--debug``) builds the same library with FA_DEBUG=1 into
_build/debug/libfa_sm100.so: every tensor-memory load, store and wait first
checks that its warp is converged (see ptx_sm100.cuh).  The binding loads it
when the environment variable FA_LIBRARY names it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa_sm100.so")
BINDING = os.path.join(HERE, "_step.so")
DEBUG_BUILD = os.path.join(BUILD, "debug")
DEBUG_LIB = os.path.join(DEBUG_BUILD, "libfa_sm100.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build")
    return path


def _deps():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "fa.h")]


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def _compile(src: str, verbose_ptxas: bool, debug: bool = False) -> str:
    obj = os.path.join(DEBUG_BUILD if debug else BUILD, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _deps()):
        cmd = [nvcc(), *ARCH, *FLAGS, *(["-DFA_DEBUG=1"] if debug else []), "-c", src, "-o", obj]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            sys.stderr.write(r.stderr)
    return obj


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def binding_abi() -> str:
    """What a build of the binding belongs to: the versions of torch (read from its
    version.py; importing it takes seconds) and of Python."""
    path = os.path.join(_torch_dir() or "", "version.py")
    version = None
    if _torch_dir() and os.path.exists(path):
        with open(path) as f:
            version = re.search(r"__version__ = ['\"]([^'\"]+)", f.read())
    return f"torch {version.group(1) if version else 'unknown'}, {sys.implementation.cache_tag}"


def _binding_lacks(torch_dir: str | None, python_include: str) -> str | None:
    """What building the binding would need and does not find here."""
    if shutil.which("g++") is None:
        return "g++"
    if torch_dir is None:
        return "torch"
    for header in (os.path.join(torch_dir, "include", "torch", "csrc", "utils", "pybind.h"),
                   os.path.join(python_include, "Python.h")):
        if not os.path.exists(header):
            return header
    return None


def _build_binding() -> str | None:
    """The Python module of csrc/py_step.cpp (it calls the library by address); None, with
    a note, where its tools are missing."""
    src = os.path.join(CSRC, "py_step.cpp")
    abi, stamp = binding_abi(), os.path.join(BUILD, "_step.abi")
    built_for = open(stamp).read() if os.path.exists(stamp) else None
    if built_for != abi or _stale(BINDING, [src, os.path.join(ROOT, "include", "fa.h")]):
        torch_dir, python_include = _torch_dir(), sysconfig.get_paths()["include"]
        lacks = _binding_lacks(torch_dir, python_include)
        if lacks:
            print(f"the Python binding of the step operators is not built: no {lacks}",
                  file=sys.stderr)
            return None
        lib, inc = os.path.join(torch_dir, "lib"), os.path.join(torch_dir, "include")
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
        paths = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), python_include,
                 os.path.join(cuda, "include")]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f'-DFA_BINDING_ABI="{abi}"',
               "-I", os.path.join(ROOT, "include"), *[f for p in paths for f in ("-isystem", p)],
               src, "-o", BINDING, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
               "-ltorch_cuda", "-ltorch_python"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
        with open(stamp, "w") as f:
            f.write(abi)
    return BINDING


def build(verbose_ptxas: bool = False, debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    os.makedirs(DEBUG_BUILD if debug else BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=len(sources) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas, debug), sources))
    if _stale(lib, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", lib, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    binding.result()                   # (raises what it failed with, behind the library)
    return lib


if __name__ == "__main__":
    print(build(verbose_ptxas="-v" in sys.argv, debug="--debug" in sys.argv))

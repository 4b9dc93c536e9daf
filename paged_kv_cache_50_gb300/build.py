"""Builds ``libpa.so`` (the C-ABI paged-attention library) in-tree with nvcc.

Every ``csrc/*.cu`` translation unit is compiled in parallel for sm_103a only
and linked into ``paged_kv_cache_50_gb300/_build/libpa.so``; the compiled
argument checks (``csrc/binding.cpp``) become the package's ``BINDING_PATH``, a file
for each torch and interpreter that they are compiled against.  Run as
``python -m paged_kv_cache_50_gb300.build`` or call :func:`build`.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libpa.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def binding_headers_missing() -> str:
    """The first header that the compiled checks need and that is not there, or
    "": libpa.so and the calls that do without the checks need neither."""
    import torch
    for h in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
              os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc",
                           "autograd", "python_variable.h")):
        if not os.path.exists(h):
            return h
    return ""


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/binding.cpp (a CPython extension over torch's headers) with
    the host compiler; returns its path."""
    from paged_kv_cache_50_gb300 import BINDING_PATH
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(BINDING_PATH) and all(
            os.path.getmtime(p) <= os.path.getmtime(BINDING_PATH) for p in deps):
        return BINDING_PATH
    import torch
    os.makedirs(OUT_DIR, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, src, "-o", tmp,
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=None, out_dir=None,
          lib_name="libpa.so") -> str:
    """Compile and link libpa.so; returns its path.  ``out_dir`` / ``lib_name``
    build a variant elsewhere (the tests' timeout variant, with its own
    defines in ``extra_flags``); the default build never includes one.  Without
    the Python or torch headers the compiled checks are left out with a warning,
    and the serving-step calls raise."""
    binding = out_dir is None
    if binding and binding_headers_missing():
        warnings.warn(f"{binding_headers_missing()} is missing: the compiled checks of the "
                      "serving-step calls are not built", RuntimeWarning, stacklevel=2)
        binding = False
    out_dir = out_dir or OUT_DIR
    lib = os.path.join(out_dir, lib_name)
    if binding:
        with cf.ThreadPoolExecutor(max_workers=1) as side:   # beside the nvcc runs
            made = side.submit(build_binding, force, verbose)
            _build_lib(lib, force, verbose, extra_flags, out_dir)
            made.result()
    else:
        _build_lib(lib, force, verbose, extra_flags, out_dir)
    return lib


def _build_lib(lib, force, verbose, extra_flags, out_dir) -> None:
    if not force and os.path.exists(lib) and all(
            os.path.getmtime(p) <= os.path.getmtime(lib) for p in _deps()):
        return
    os.makedirs(out_dir, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])
    objs = []
    cmds = []
    for src in _sources():
        obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmds.append([cc, *ARCH, *flags, "-c", src, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    with cf.ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 4)) as ex:
        list(ex.map(run, cmds))
    tmp = lib + f".{os.getpid()}.tmp"
    run([cc, *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs])
    os.replace(tmp, lib)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
    print(LIB)

"""Build libmla.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and
_calls.so (the compiled part of the Python binding) with g++.

Each ``csrc/*.cu`` compiles to an object in ``_build/`` in parallel, then the
objects link into ``mla_paged_kv_concat_gb300/libmla.so``; ``csrc/bind.cpp``
compiles beside them and links against it and torch, and is made anew for
another torch or Python.  ptxas resource usage
(``-Xptxas -v``) goes to ``_build/ptxas.log``.  Run ``python -m
mla_paged_kv_concat_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmla.so")
BIND = os.path.join(PKG, "_calls.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-Xptxas", "-v", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(out: str, deps) -> bool:
    """Whether ``out`` is there and no older than any of ``deps``."""
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__])


def _bind_versions() -> str:
    """What the binding is compiled for; another torch or Python cannot load
    it, or reads its tensors wrongly."""
    import importlib.metadata as md
    try:
        torch = md.version("torch")
    except md.PackageNotFoundError:
        torch = "none"
    return f"torch {torch}, {sys.implementation.cache_tag}, {platform.machine()}\n"


def _bind_stamp() -> str:
    return os.path.join(BUILD, os.path.basename(BIND) + ".versions")


def _bind_up_to_date() -> bool:
    try:
        with open(_bind_stamp()) as f:
            if f.read() != _bind_versions():
                return False
    except OSError:
        return False
    return _newer(BIND, [BIND_SRC, __file__] + glob.glob(os.path.join(ROOT, "include", "*.h")))


def up_to_date() -> bool:
    return _lib_up_to_date() and _bind_up_to_date()


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def _compile_bind() -> str:
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "bind.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", BIND_SRC, "-o", obj,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for inc in (os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")):
        cmd += ["-isystem", inc]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_bind(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", "-L" + lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)


def _link_lib(objs) -> None:
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libmla.so", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what changed; returns the path of libmla.so.

    The library needs neither torch nor the binding: it is linked first, and
    what goes wrong with the binding is raised after that.
    """
    lib, bind = force or not _lib_up_to_date(), force or not _bind_up_to_date()
    if not lib and not bind:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        bind_obj = ex.submit(_compile_bind) if bind else None
        results = list(ex.map(_compile, srcs)) if lib else []
    if lib:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            for (obj, log), src in zip(results, srcs):
                f.write(f"==== {os.path.basename(src)}\n{log}\n")
        _link_lib([o for o, _ in results])
    if bind:
        obj = bind_obj.result()
        if os.path.exists(_bind_stamp()):
            os.remove(_bind_stamp())  # no stamp beside a binding that is not its own
        _link_bind(obj)
        with open(_bind_stamp(), "w") as f:
            f.write(_bind_versions())
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)

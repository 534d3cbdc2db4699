"""Builds libtld_gb300.so from csrc/ with nvcc for sm_103a, and with g++ the Python module that marshals
its short calls (in-tree, _build/)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libtld_gb300.so")
# debug build: the kernels' index checks compiled in (TLD_DEBUG_CHECKS)
DEBUG_LIB = os.path.join(BUILD, "libtld_gb300_debug.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
          "-I", INCLUDE]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    extra = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return sources() + extra + [os.path.join(INCLUDE, "dec.h")]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_calls(force: bool = False) -> str | None:
    """Compiles csrc/py_calls.cpp against this Python and this torch; None, with a warning, where their headers are
    missing: the library does not need it."""
    import sysconfig

    try:
        import torch

        from . import dec
        out = dec.calls_path()
        includes = [os.path.join(os.path.dirname(torch.__file__), "include"), sysconfig.get_paths()["include"]]
        needed = [os.path.join(includes[0], "torch", "csrc", "autograd", "python_variable.h"),
                  os.path.join(includes[1], "Python.h")]
        missing = [p for p in needed if not os.path.exists(p)]
    except ImportError as e:
        missing = [str(e)]
    if missing:
        warnings.warn(f"a decode step's calls will be marshalled in Python: {', '.join(missing)} is missing", RuntimeWarning)
        return None
    src = os.path.join(CSRC, "py_calls.cpp")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "dec.h")))
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    os.makedirs(BUILD, exist_ok=True)
    tmp = out + f".{os.getpid()}.tmp"
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for p in includes for x in ("-I", p)), "-I", os.path.join(includes[0], "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", INCLUDE, src, "-o", tmp,
           "-L", libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          debug: bool = False) -> str:
    """Compile every .cu in csrc/ in parallel and link the shared library (with
    debug=True: the debug build, index checks compiled in, in its own objects)."""
    lib = DEBUG_LIB if debug else LIB
    if not force and not ptxas_info and up_to_date(lib):
        build_calls()
        return lib
    objdir = os.path.join(BUILD, "debug") if debug else BUILD
    os.makedirs(objdir, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    if debug:
        extra.append("-DTLD_DEBUG_CHECKS")

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 4)) as ex:
        calls = ex.submit(build_calls, force)
        objs = list(ex.map(compile_one, sources()))
        calls.result()
    tmp = lib + f".{os.getpid()}.tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv,
                debug="--debug" in sys.argv))

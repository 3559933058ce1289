"""Builds libkvpaged.so in-tree with nvcc for sm_103a (no cmake), and beside it
the Python binding's extension module.

Each .cu (and host-only .cpp) file is compiled in parallel to an object, then linked into
paged_kv_cache_125_gb300/_build/libkvpaged.so.  A rebuild happens only when a
source or header is newer than the library.

The extension module (csrc/python/calls.cpp) is host code against the C++
headers of the installed torch, compiled with g++ next to the nvcc jobs; its
file name carries that torch's version.  The library needs none of these: without
torch there is no extension module to build, and where it cannot be built a
warning says why and the Python binding makes the same calls through ctypes.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libkvpaged.so")
CALLS_SRC = os.path.join(CSRC, "python", "calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvpaged")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def calls_path() -> str:
    import torch
    return os.path.join(OUT, "_kvpaged_calls_%s.so" % re.sub(r"\W", "_", torch.__version__))


def _newer(deps, out: str) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(d) > os.path.getmtime(out) for d in deps)


def _stale() -> bool:
    return _newer(sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__], LIB)


def _calls_stale(force: bool = False) -> bool:
    try:
        out = calls_path()
    except ImportError:
        return False  # no torch: nothing to bind to
    return force or _newer([CALLS_SRC, os.path.join(INCLUDE, "kvpaged.h"), __file__], out)


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_calls() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(OUT, "calls_py.o")
    _run(["g++", "-c", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", CALLS_SRC, "-o", obj, "-I", INCLUDE,
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
          "-isystem", sysconfig.get_paths()["include"]], "g++ for calls.cpp")
    return obj


def _link_calls(obj: str):
    import torch
    tmp = calls_path() + f".tmp{os.getpid()}"
    _run(["g++", "-shared", obj, "-o", tmp, "-L" + OUT, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python"], "link of the extension module")
    os.replace(tmp, calls_path())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OUT, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_compile_calls) if _calls_stale(force) else None
        _build_library(force, verbose, extra_flags)
        if calls is not None:
            try:
                _link_calls(calls.result())
            except (RuntimeError, OSError, ImportError) as e:
                if os.path.exists(calls_path()):  # of an older header: its calls may not match the library's
                    os.remove(calls_path())
                warnings.warn(f"the extension module was not built, its calls go through ctypes: {e}")
    return LIB


def _build_library(force: bool, verbose: bool, extra_flags) -> str:
    if not force and not _stale():
        return LIB
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"] + list(extra_flags)
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc(), "-c", src, "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc(), "-shared", "-o", tmp] + objs + ARCH, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))

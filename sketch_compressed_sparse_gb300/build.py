"""Build libs2.so (the sm_103a kernels and the C ABI) in-tree with nvcc.

Each .cu file compiles to an object in parallel, then nvcc links the shared
library into ``sketch_compressed_sparse_gb300/_lib/libs2.so``. Where Python's
headers and a host compiler are installed, ``_s2calls`` (a shorter way from
Python to the 8-bit layer's calls) is built beside it. Each is skipped where
it is newer than its sources and headers.

Usage: ``python -m sketch_compressed_sparse_gb300.build [--force] [--verbose]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "_lib")
OBJDIR = os.path.join(LIBDIR, "obj")
LIB = os.path.join(LIBDIR, "libs2.so")
CALLS_SRC = os.path.join(CSRC, "s2_calls.cpp")
CALLS = os.path.join(LIBDIR, "_s2calls" + sysconfig.get_config_var("EXT_SUFFIX"))
HEADER = os.path.join(ROOT, "include", "s2.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libs2")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _python_headers():
    """Directory of Python.h, or None."""
    inc = sysconfig.get_paths()["include"]
    return inc if os.path.exists(os.path.join(inc, "Python.h")) else None


def header_flags():
    """Says in a binary which s2.h it was compiled from: the extension is used only with a library of the same."""
    with open(HEADER, "rb") as f:
        return [f"-DS2_HEADER_ID=h{hashlib.sha256(f.read()).hexdigest()[:16]}"]


def _older(target, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in deps)


def _stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER])


def _calls_stale() -> bool:
    return _python_headers() is not None and _older(CALLS, [CALLS_SRC, os.path.join(CSRC, "s2_header_id.h"), HEADER])


def _build_calls() -> None:
    inc = _python_headers()
    if not inc:
        return
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", inc,
           "-I", os.path.join(ROOT, "include"), *header_flags(), CALLS_SRC, "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = "" if r.returncode == 0 else r.stdout + r.stderr or f"{cmd[0]} failed"
    except OSError as e:
        log = str(e)
    if log:  # ctypes makes the calls then
        print(f"_s2calls was not built: {log}", file=sys.stderr)
        for p in (tmp, CALLS):
            if os.path.exists(p):
                os.remove(p)
        return
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every kernel for sm_103a and link libs2.so; returns its path."""
    if not force and not _stale():
        if _calls_stale():
            _build_calls()
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *header_flags(), *extra, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_build_calls)
        results = list(ex.map(compile_one, sources()))
        calls.result()
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
                ptxas_info="--ptxas-info" in sys.argv))

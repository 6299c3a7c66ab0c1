"""Build the in-tree shared library ``libmoedecode.so`` (sm_100a) with nvcc.

Usage: ``python -m mixture_experts_decode_gemv_b200.build [--force] [--ptxas-verbose]``.
The library is rebuilt only when a source or header is newer than it (or with ``--force``).
"""
from __future__ import annotations

import argparse
from concurrent.futures import ThreadPoolExecutor
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoedecode.so")

SOURCES = ["api.cu", "host_formats.cpp", "no_alloc.cu", "route_rows.cu", "quantize_rows.cu",
           "matmul_int8.cu", "combine_rows.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoedecode.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)
             if f.endswith((".cu", ".cuh", ".cpp", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _object_up_to_date(obj: str, dep: str) -> bool:
    """Whether ``obj`` is newer than every file its dependency list names."""
    if not (os.path.exists(obj) and os.path.exists(dep)):
        return False
    text = open(dep).read().replace("\\\n", " ")
    files = text.split(":", 1)[1].split()
    t = os.path.getmtime(obj)
    return all(os.path.exists(f) and os.path.getmtime(f) <= t
               for f in files + [os.path.abspath(__file__)])


def _run(cmd, quiet: bool, verbose: bool) -> None:
    if not quiet:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, cwd=CSRC, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose or (res.stderr.strip() and not quiet):
        print(res.stderr, file=sys.stderr)


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False,
          defines=(), out: str = None) -> str:
    """Compile the library; ``defines`` (e.g. ``("MOE_PHASE_TIMERS",)``) and ``out`` give a
    separately named variant build. Sources compile in parallel, and one whose object is newer
    than everything it includes is not compiled again."""
    target = out or LIB
    if not force and not defines and out is None and up_to_date():
        return LIB
    variant = "-".join(defines) or "default"
    objdir = os.path.join(PKG, "_build", "".join(c if c.isalnum() or c in "-_" else "_"
                                                 for c in variant))
    os.makedirs(objdir, exist_ok=True)
    flags = ["-O3", "-std=c++17", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
             "--expt-relaxed-constexpr", "-I", INCLUDE, *[f"-D{d}" for d in defines]]
    if ptxas_verbose:
        flags = ["-Xptxas", "-v", *flags]

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src + ".o")
        dep = obj + ".d"
        if force or not _object_up_to_date(obj, dep):
            _run([_nvcc(), *flags, "-MD", "-MF", dep, "-c", os.path.join(CSRC, src), "-o",
                  obj + ".tmp.o"], quiet, ptxas_verbose)
            os.replace(obj + ".tmp.o", obj)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
        objects = list(pool.map(compile_one, SOURCES))
    _run([_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", target + ".tmp", *objects], quiet,
         False)
    os.replace(target + ".tmp", target)
    return target


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    ap.add_argument("--define", action="append", default=[])
    ap.add_argument("--out", default=None)
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_verbose, defines=a.define, out=a.out))

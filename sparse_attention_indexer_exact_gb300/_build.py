"""Build step for libgvrtopk.so (the CUDA kernels and their C ABI), in-tree, for sm_103a.

``build_library()`` runs nvcc over each translation unit (``csrc/gvr_topk.cu``,
``csrc_cache/*.cu``) at the same time, links them, and writes ``libgvrtopk.so``
beside this file; it rebuilds only when a source is newer than the library.  No
CMake, no torch extension machinery: the library is a plain shared object with
an ``extern "C"`` interface (``include/gvr_topk.h``, ``include/gvr_cache.h``).
"""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile
import threading
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_CACHE = os.path.join(PKG, "csrc_cache")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libgvrtopk.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
_lock = threading.Lock()


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted([f for d in (CSRC, CSRC_CACHE) for ext in ("*.cu", "*.cuh", "*.h") for f in glob.glob(os.path.join(d, ext))] +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def units() -> list[str]:
    """The translation units."""
    return [f for f in sources() if f.endswith(".cu")]


def compile_command(unit: str, out: str, extra=()) -> list[str]:
    return [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, *extra,
            "-c", unit, "-o", out]


def link_command(objects: list[str], out: str = LIB_PATH) -> list[str]:
    return [nvcc_path(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objects, "-o", out]


def _run(cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def stale(out: str = LIB_PATH) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in sources())


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile libgvrtopk.so for sm_103a if it is missing or older than its sources."""
    with _lock:
        if force or stale():
            extra = ["-Xptxas", "-v"] if verbose else []
            with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor() as pool:
                jobs = [(u, os.path.join(tmp, os.path.basename(u) + ".o")) for u in units()]
                said = list(pool.map(lambda j: _run(compile_command(*j, extra)), jobs))
                said.append(_run(link_command([o for _, o in jobs])))
            if verbose:
                print("".join(said))
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))

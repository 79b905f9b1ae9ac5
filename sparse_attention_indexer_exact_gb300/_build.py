"""Build step for libgvrtopk.so (the CUDA kernels and their C ABI), in-tree, for sm_103a.

``build_library()`` runs nvcc over each translation unit (``csrc/gvr_topk.cu``,
``csrc_cache/*.cu``) at the same time, links them, and writes ``libgvrtopk.so``
beside this file; it rebuilds only when a source is newer than the library.  No
CMake, no torch extension machinery: the library is a plain shared object with
an ``extern "C"`` interface (``include/gvr_topk.h``, ``include/gvr_cache.h``).
Beside it g++ builds ``_native.so`` (``_native.cpp``), the short way from torch
tensors to the cache's calls, against the installed torch and the library.  The
library does not need it, or torch: where those or Python's headers are not
there, ``_native.so`` is left out with a warning, and the cache's calls go through
ctypes.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import tempfile
import threading
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_CACHE = os.path.join(PKG, "csrc_cache")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libgvrtopk.so")
NATIVE_SOURCE = os.path.join(PKG, "_native.cpp")
NATIVE_PATH = os.path.join(PKG, "_native.so")
NATIVE_STAMP = NATIVE_PATH + ".for"  # the torch and Python that it was built for
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


def _torch_root() -> str | None:
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def native_target() -> str:
    """The torch and Python of this process: _native.so is compiled against their insides, so it fits no others."""
    torch = _torch_root()
    version = "none"
    if torch is not None:
        scope: dict = {}
        with open(os.path.join(torch, "version.py")) as f:  # without importing torch
            exec(f.read(), scope)
        version = str(scope["__version__"])
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}"


def native_stale() -> bool:
    if stale(NATIVE_PATH, [NATIVE_SOURCE, *glob.glob(os.path.join(INCLUDE, "*.h"))]) or not os.path.exists(NATIVE_STAMP):
        return True
    with open(NATIVE_STAMP) as f:
        return f.read() != native_target()


def native_lacks() -> str | None:
    """What _native.so cannot be built without and is not there."""
    torch = _torch_root()
    if torch is None:
        return "torch is not installed"
    for header in (os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return f"{header} is missing"
    return None if shutil.which("g++") else "g++ is missing"


def native_commands(obj: str, out: str = NATIVE_PATH) -> tuple[list[str], list[str]]:
    """Compiling and linking the tensor binding (the link needs libgvrtopk.so)."""
    torch = _torch_root()
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include") if os.path.isabs(nvcc_path()) else \
        "/usr/local/cuda/include"
    include = [os.path.join(torch, "include"), sysconfig.get_paths()["include"], cuda, INCLUDE]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f'-DGVR_BUILT_FOR="{native_target()}"', *[x for d in include for x in ("-I", d)], "-c",
                NATIVE_SOURCE, "-o", obj]
    link = ["g++", "-shared", obj, "-o", out, "-L", PKG, "-l:libgvrtopk.so", "-L", os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def stale(out: str = LIB_PATH, of: list[str] | None = None) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in (of or sources()))


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile libgvrtopk.so for sm_103a, and _native.so where it can be built, if missing or older than their sources
    (_native.so: or built for another torch or Python)."""
    with _lock:
        library = force or stale()
        native = force or library or native_stale()
        lacks = native_lacks() if native else None
        if lacks:
            native = False
            warnings.warn(f"_native.so is not built ({lacks}): the cache calls go through ctypes", RuntimeWarning)
        if library or native:
            extra = ["-Xptxas", "-v"] if verbose else []
            with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor() as pool:
                jobs = [(u, os.path.join(tmp, os.path.basename(u) + ".o")) for u in units()] if library else []
                compiled = [pool.submit(_run, compile_command(*j, extra)) for j in jobs]
                if native:
                    native_compile, native_link = native_commands(os.path.join(tmp, "native.o"))
                    native_compiled = pool.submit(_run, native_compile)
                said = [c.result() for c in compiled]
                if library:
                    said.append(_run(link_command([o for _, o in jobs])))
                if native:  # behind the library, which is there whatever becomes of this
                    said.append(native_compiled.result())
                    if os.path.exists(NATIVE_STAMP):
                        os.remove(NATIVE_STAMP)
                    said.append(_run(native_link))
                    with open(NATIVE_STAMP, "w") as f:
                        f.write(native_target())
            if verbose:
                print("".join(said))
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))

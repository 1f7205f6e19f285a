"""Builds the CUDA library in-tree for sm_103a with plain nvcc (no CMake).

Each .cu translation unit is compiled in parallel, then linked into
``paged_mla_speculative_tree_gb300/_lib/libmla_tree_verify.so``.  Beside it g++ makes
the Python extension through which some of its entries are called; it needs the
headers of Python and torch, and without them the library is built all the same.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libmla_tree_verify.so")
EXT_SRC = os.path.join(CSRC, "binding_ext.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]
CXX = "g++"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _abi():
    return [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]


def _current(made, sources) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(d) <= os.path.getmtime(made) for d in sources)


def _library_current() -> bool:
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return _current(LIB, sources() + headers + _abi())


def _extension_current() -> bool:
    return _current(extension_path(), [EXT_SRC] + _abi())


def up_to_date() -> bool:
    return _library_current() and _extension_current()


def extension_path() -> str:
    """The extension for this torch and this Python, whose layouts are compiled into it."""
    import torch
    return os.path.join(OUT_DIR, f"binding_ext.torch-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _run(what, cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r


def _build_extension() -> None:
    torch_dir = list(importlib.util.find_spec("torch").submodule_search_locations)[0]
    path = extension_path()
    obj, tmp = os.path.join(BUILD_DIR, "binding_ext.o"), path + f".tmp{os.getpid()}"
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include")]
    _run(f"{CXX} on {EXT_SRC}", [CXX, "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in inc), "-c", EXT_SRC, "-o", obj])
    _run("link", [CXX, "-shared", "-o", tmp, obj, "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(tmp, path)


def _build_library(ex, verbose, extra) -> None:
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        r = _run(f"nvcc on {src}", [cc, *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj])
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    tmp = LIB + f".tmp{os.getpid()}"
    _run("link", [cc, *ARCH, "-shared", "-o", tmp, *ex.map(compile_one, sources())])
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Builds what is missing or older than its sources; returns the library's path.  An extension that could not be
    built is reported on stderr: the calls that go through it raise, all others need only the library."""
    library, extension = force or not _library_current(), force or not _extension_current()
    if not library and not extension:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(sources()) + 1, os.cpu_count() or 4)) as ex:
        made = ex.submit(_build_extension) if extension else None
        if library:
            _build_library(ex, verbose, extra)
        try:
            if made:
                made.result()
        except (RuntimeError, OSError) as e:  # no headers, no compiler
            sys.stderr.write(f"the extension was not built: {e}\n")
            if os.path.exists(extension_path()):
                os.remove(extension_path())  # of other sources
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

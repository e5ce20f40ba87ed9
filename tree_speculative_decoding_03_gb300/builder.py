"""Builds libtsv.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel into `_build/`, then the objects are
linked into `_build/libtsv.so` (static CUDA runtime, so the library needs no
runtime search path).  Rebuilds only when a source or header is newer than the
library.  The serving operators' argument marshalling (`binding/marshal.cpp`, against torch's
headers) is compiled beside it with the host compiler into `_build/`, under a name that holds the
Python ABI and the torch version it belongs to; without torch's or Python's headers it is left out.
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import warnings
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libtsv.so")
MARSHAL_SRC = os.path.join(HERE, "binding", "marshal.cpp")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{INCLUDE}", "--expt-relaxed-constexpr"]


def _sources():
    # CUDA translation units (those of the serving operators in their own folder) and the
    # host-only C++ ones (tree construction)
    return sorted(p for pat in ("*.cu", "*.cpp", "serving/*.cu") for p in glob.glob(os.path.join(CSRC, pat)))


def _deps():
    headers = [p for pat in ("*.cuh", "serving/*.cuh") for p in glob.glob(os.path.join(CSRC, pat))]
    return _sources() + headers + glob.glob(os.path.join(INCLUDE, "*.h"))


# Test builds of the same sources: "checked" adds device-side index checks
# (-DTSV_CHECKED), "hooks" shortens the bounded waits and adds a stall switch and a limit on the plan's cluster
# (-DTSV_TEST_HOOKS).  Each is built into its own folder; the product library is the
# default (no variant).
VARIANT_FLAGS = {"checked": ["-DTSV_CHECKED"], "hooks": ["-DTSV_TEST_HOOKS"]}


def lib_path(variant=None) -> str:
    return LIB if variant is None else os.path.join(OUT_DIR, variant, "libtsv.so")


def up_to_date(variant=None) -> bool:
    lib = lib_path(variant)
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build_library(verbose: bool = False, extra_flags=(), variant=None) -> str:
    lib = lib_path(variant)
    extra_flags = list(extra_flags) + VARIANT_FLAGS.get(variant, [])
    if up_to_date(variant) and not (extra_flags and variant is None):
        return lib
    out_dir = os.path.dirname(lib)
    os.makedirs(out_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def marshal_path() -> str:
    """Where the argument marshalling of this Python and this torch lies: one built against
    another torch is never loaded, however new the file."""
    import sysconfig

    import torch
    tag = f"{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}"
    return os.path.join(OUT_DIR, "_marshal." + re.sub(r"[^A-Za-z0-9_.-]", "_", tag) + ".so")


def _marshal_includes() -> list:
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or "/usr/local/cuda/bin/nvcc")))
    return [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(cuda, "include")]


def marshal_missing() -> Optional[str]:
    """What the argument marshalling needs and does not find (None: nothing)."""
    try:
        dirs = _marshal_includes()
    except ImportError:
        return "torch"
    for name in ("Python.h", "torch/csrc/autograd/python_variable.h", "c10/cuda/CUDAStream.h", "cuda_runtime_api.h"):
        if not any(os.path.exists(os.path.join(d, name)) for d in dirs):
            return name
    return None


def build_marshal() -> Optional[str]:
    """Compiles the argument marshalling of the serving operators (host code).  Where torch or a
    header is missing the rest of the package stands without it: a warning, and those operators
    raise when they are called."""
    missing = marshal_missing()
    if missing is not None:
        warnings.warn(f"{missing} not found: the serving operators' binding is not built", RuntimeWarning)
        return None
    import torch
    out = marshal_path()
    deps = [MARSHAL_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
        return out
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           *(f"-isystem{d}" for d in [*_marshal_includes(), INCLUDE]), MARSHAL_SRC, "-o", tmp,
           f"-L{os.path.join(os.path.dirname(torch.__file__), 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {os.path.basename(MARSHAL_SRC)} failed:\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build_library(verbose=True))
    print(build_marshal())

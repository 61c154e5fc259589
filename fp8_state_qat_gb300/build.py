"""Compile the CUDA library ``libgdnqat.so`` in-tree for sm_103a, and the Python extension
``gdnqat_layer.so`` (csrc/layer_ext.cpp, g++ against torch's headers) beside it.

Each ``csrc/*.cu`` is compiled to an object in parallel (one ``-gencode``, no cmake), then
linked into ``fp8_state_qat_gb300/_lib/libgdnqat.so`` with the CUDA runtime linked
statically. Rebuilds only when a source or header is newer than the library.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libgdnqat.so")
EXT_SOURCE = os.path.join(CSRC, "layer_ext.cpp")
EXT_PATH = os.path.join(LIB_DIR, "gdnqat_layer.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return p


def _sources(csrc=CSRC):
    return sorted(glob.glob(os.path.join(csrc, "*.cu")))


def headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [
        os.path.join(ROOT, "include", "gdnqat.h"), __file__]


def _deps():
    return _sources() + headers()


def newer_than(out: str, deps) -> bool:
    """`out` exists and no file in `deps` was modified after it."""
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps)


def _ext_deps():
    return [EXT_SOURCE, os.path.join(ROOT, "include", "gdnqat.h"), __file__]


def up_to_date() -> bool:
    return newer_than(LIB_PATH, _deps())


def compile_extension(out: str = EXT_PATH) -> str:
    """g++ the argument checks and allocations of layer.py against this Python and this torch."""
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    os.makedirs(os.path.dirname(out), exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden", *[f"-isystem{d}" for d in include],
           "-I", sysconfig.get_paths()["include"], EXT_SOURCE, "-o", tmp, "-L" + os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + os.path.join(cuda, "lib64"), "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(EXT_SOURCE)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def compile_library(sources, out: str, obj_dir: str, verbose: bool = False) -> str:
    """nvcc each of `sources` (objects in `obj_dir`, in parallel) and link them into the shared
    library `out` with the CUDA runtime linked statically. A source is a path, or a pair
    (path, extra -D macros for that file)."""
    os.makedirs(obj_dir, exist_ok=True)
    os.makedirs(os.path.dirname(out), exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                    "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(item):
        src, defines = (item, ()) if isinstance(item, str) else item
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *flags, *[f"-D{d}" for d in defines], "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, sources))
    if verbose:
        for _, log in results:
            print(log)
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu into libgdnqat.so (skipped when it is up to date)."""
    if not force and up_to_date():
        return LIB_PATH
    return compile_library(_sources(), LIB_PATH, OBJ_DIR, verbose=verbose)


def build_extension(force: bool = False) -> str:
    """Compile csrc/layer_ext.cpp into gdnqat_layer.so (skipped when it is up to date). Only the operators of
    layer.py need it."""
    if not force and newer_than(EXT_PATH, _ext_deps()):
        return EXT_PATH
    return compile_extension(EXT_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and the extension, side by side."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(build_extension, force)
        build_library(force, verbose)
        ext.result()
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

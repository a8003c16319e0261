"""Build libpagedkv.so in-tree with nvcc for sm_100a.

    python -m paged_kv_cache_462_b200.build [--force]

Each .cu file compiles to an object in parallel; the objects link into
``paged_kv_cache_462_b200/libpagedkv.so`` (the CUDA runtime linked statically). The binding's
hot path, ``csrc/fastcall.cpp``, becomes the extension module ``_fastcall`` beside it, for the Python and
torch that build it; the package works without it, only slower, so that a failure there is a warning.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libpagedkv.so")
FASTCALL = os.path.join(HERE, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))   # one file a Python
BUILD_DIR = os.path.join(HERE, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _newer(target, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def torch_version() -> str:
    """The installed torch's version ("" without one), as its package metadata has it."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return ""


def build_fastcall(force: bool = False) -> str:
    """The extension module _fastcall (g++, torch's and Python's headers). Rebuilt for another torch: the
    version it was built for stands in a file beside the objects, and in the module."""
    src = os.path.join(CSRC, "fastcall.cpp")
    stamp = os.path.join(BUILD_DIR, os.path.basename(FASTCALL) + ".torch")
    version = torch_version()
    spec = importlib.util.find_spec("torch")
    if not version or spec is None:
        raise RuntimeError("_fastcall needs torch's headers")
    if not force and _newer(FASTCALL, [src, os.path.join(INCLUDE, "pkv.h")]) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == version:
                return FASTCALL
    os.makedirs(BUILD_DIR, exist_ok=True)
    torch_dir = list(spec.submodule_search_locations)[0]
    tmp = FASTCALL + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
           f'-DPKV_TORCH_VERSION="{version}"', "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(torch_dir, "include"),
           "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), src,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FASTCALL)
    with open(stamp, "w") as f:
        f.write(version)
    return FASTCALL


def build(force: bool = False, verbose: bool = False, strict: bool = False) -> str:
    """The library, then the extension module; `strict` raises where that one cannot be built."""
    build_library(force, verbose)
    try:
        build_fastcall(force)
    except (OSError, RuntimeError) as e:
        if strict:
            raise
        print(f"warning: built without the binding's hot path: {e}", file=sys.stderr)
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))

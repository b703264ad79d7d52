"""Builds libttt_b200.so in-tree from csrc/*.cu for sm_100a with nvcc.

    python -m linear_attention_ttt_b200.build [--force] [--verbose] [--debug-bounds]

--debug-bounds builds libttt_b200_dbg.so instead (objects under csrc/_build_dbg/),
compiled with -DTTT_DEBUG_BOUNDS: the kernels check their index arithmetic
and report a failed check as TTT_ERR_BOUNDS through ttt_get_device_status.

Each translation unit is compiled to an object under csrc/_build/ and the
objects are linked into linear_attention_ttt_b200/libttt_b200.so (cudart
linked statically, so the library shares the CUDA driver context of whatever
process loads it). A unit is rebuilt when it, or any header it may include,
is newer than its object. csrc/binding.cpp, the native half of the Python
binding, is compiled with g++ against torch's headers into
linear_attention_ttt_b200/_binding.so.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(CSRC, "_build")
LIB = os.path.join(PKG, "libttt_b200.so")
BUILD_DBG = os.path.join(CSRC, "_build_dbg")
LIB_DBG = os.path.join(PKG, "libttt_b200_dbg.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O3", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def binding_key() -> str:
    """What _binding.so is compiled against: torch, its C++ ABI and Python's."""
    import sysconfig

    import torch
    return (f"torch {torch.__version__} {torch.version.git_version} "
            f"cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python {sysconfig.get_config_var('EXT_SUFFIX')}")


def build_binding(force: bool = False) -> str:
    """_binding.so (see csrc/binding.cpp). Only torch's headers and libraries are used. It is
    built again when its source or what it is compiled against has changed."""
    newest = max(os.path.getmtime(f) for f in (BINDING_SRC, os.path.join(ROOT, "include", "ttt.h")))
    key, stamp = binding_key(), os.path.join(BUILD, "binding.key")
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == key:
                return BINDING
    import sysconfig

    import torch
    os.makedirs(BUILD, exist_ok=True)
    if os.path.exists(stamp):
        os.remove(stamp)
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(base, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DTTT_BUILT_FOR="{key}"',
           *(f"-I{i}" for i in inc), BINDING_SRC, "-o", BINDING, f"-L{lib}", f"-Wl,-rpath,{lib}",
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed on binding.cpp")
    with open(stamp, "w") as f:
        f.write(key)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra=(), debug_bounds: bool = False) -> str:
    build_binding(force)
    build_dir, lib = (BUILD_DBG, LIB_DBG) if debug_bounds else (BUILD, LIB)
    if debug_bounds:
        extra = (*extra, "-DTTT_DEBUG_BOUNDS")
    os.makedirs(build_dir, exist_ok=True)
    hdr_time = max([os.path.getmtime(h) for h in _headers()] + [0])
    objs, stale = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj)
                and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_time)):
            continue
        stale.append((src, obj))

    def compile_unit(unit):
        src, obj = unit
        cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")

    with ThreadPoolExecutor(max(1, os.cpu_count() or 1)) as pool:  # a unit takes up to minutes
        list(pool.map(compile_unit, stale))
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(lib) or os.path.getmtime(lib) < newest:
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", *objs, "-o", lib, "-lcuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--debug-bounds", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose, debug_bounds=args.debug_bounds))

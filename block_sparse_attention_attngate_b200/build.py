"""Build libseer.so (sm_100a) in-tree with nvcc, and the Python call layer _seer_call.*.so beside it.

    python -m block_sparse_attention_attngate_b200.build [--force] [--verbose]

Each csrc/*.cu compiles to an object under _build/, then everything links
into block_sparse_attention_attngate_b200/libseer.so with the CUDA runtime
linked statically (the library does not depend on which libcudart a host
process loaded).  csrc/binding.cpp, which checks tensors for the binding,
compiles against torch's headers with g++; the Python and the torch that it
was compiled for are in its file's name, and where it cannot be built the
binding does without.  A rebuild happens only when a source or header is
newer than what is built from it.
"""

from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libseer.so")
CALL_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
         "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def call_layer_path() -> str:
    """The call layer's file for this Python and this torch: it uses the C++ interfaces of both."""
    import torch
    return os.path.join(PKG, f"_seer_call.{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def build_call_layer(force: bool = False, verbose: bool = False) -> str:
    import torch
    path = call_layer_path()
    deps = [CALL_SRC, os.path.join(INCLUDE, "seer.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in deps):
        return path
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [os.path.join(os.path.dirname(torch.__file__), "include"), sysconfig.get_paths()["include"], cuda]
    tmp = path + ".tmp"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for i in includes for x in ("-isystem", i)], "-I", INCLUDE, CALL_SRC, "-o", tmp, "-L", lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    lib = build_library(force, verbose, ptxas_info)
    try:
        build_call_layer(force, verbose)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the compiled call layer was not built, calls around the decode step take longer on the host: {e}",
                      RuntimeWarning, stacklevel=2)
    return lib


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if (verbose or ptxas_info) and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-ldl"]   # the static CUDA runtime (nvcc default) needs libdl
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / shared memory")
    a = ap.parse_args(argv)
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose, ptxas_info=a.ptxas_info))


if __name__ == "__main__":
    sys.exit(main())

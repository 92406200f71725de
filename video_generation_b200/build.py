"""Build libaf.so (the CUDA library behind include/af.h) for sm_100a with nvcc, and
_binding.so (csrc/binding.cpp, the operators' tensor marshalling) with g++.

Usage: python -m video_generation_b200.build [--force]
The library is written in-tree as video_generation_b200/libaf.so; objects go to
_build/ at the repository root.  Rebuilds only what changed.
"""
from __future__ import annotations

import argparse
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
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libaf.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["af_api.cu", "af_kernels.cu", "af_gemm_tc.cu", "af_attn_tc.cu", "af_noalloc.cu", "af_qk.cu", "af_cache4.cu",
           "af_attn4_tc.cu", "af_ops.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list:
    hdr = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hdr + [os.path.join(INCLUDE, "af.h"), os.path.abspath(__file__)]


def _stale(target: str, deps: list) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _binding_lacks(torch) -> str | None:
    """What this machine lacks for the binding, or None.  libaf.so needs none of it."""
    if torch is None or not os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")):
        return "PyTorch with CUDA"
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None


def _build_binding(cuda: str, force: bool, verbose: bool) -> None:
    """Builds _binding.so; where that is impossible it is left out (the operators' Python calls then say so), and the
    library still serves C callers and the other Python calls."""
    torch = _torch_dir()
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(INCLUDE, "af.h"), os.path.abspath(__file__)]
    if torch:
        deps.append(os.path.join(torch, "version.py"))
    if not force and not _stale(BINDING, deps):
        return
    lacks = _binding_lacks(torch)
    if lacks:
        if os.path.exists(BINDING):
            os.remove(BINDING)   # of other sources
        sys.stderr.write(f"_binding.so not built: it needs {lacks}\n")
        return
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + os.path.join(torch, "include"),
           "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I" + os.path.join(cuda, "include"),
           "-I" + sysconfig.get_paths()["include"], src, "-o", BINDING + ".new", "-L" + os.path.join(torch, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("g++ failed on binding.cpp")
    os.replace(BINDING + ".new", BINDING)


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()
    hdrs = _deps()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [cc, *ARCH, *FLAGS, *(extra or []), "-c", s, "-o", o]
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if force or jobs or _stale(LIB, objs):
        cmd = [cc, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libaf.so failed")
    _build_binding(os.path.dirname(os.path.dirname(os.path.realpath(cc))), force, verbose)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills per kernel")
    a = ap.parse_args()
    ex = ["-Xptxas", "-v"] if a.ptxas_info else None
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra=ex))

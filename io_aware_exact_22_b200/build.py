"""Builds libfa.so in-tree (io_aware_exact_22_b200/libfa.so) with nvcc for sm_100a, and the
debug build libfa_debug.so (the same sources with FA_DEBUG: device-side index checks and tile
visit counters, see include/fa.h).

    python -m io_aware_exact_22_b200.build [--force] [--verbose] [--debug | --all]

libfa.so comes with _fa_torch.so, the extension of the binding (csrc/fa_torch.cpp, host code only,
compiled against the torch that runs the build; without torch the build says so and makes the library
alone).

Each .cu file under csrc/ is compiled to an object in _build/ (skipped when the object is
newer than every source and header), then linked into one shared library against the static
CUDA runtime.  The tensor-map encoder is fetched from the driver at run time, so the library
does not link libcuda.
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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfa.so")
BUILD_DEBUG = os.path.join(ROOT, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libfa_debug.so")

EXT_SRC = os.path.join(CSRC, "fa_torch.cpp")
EXT = os.path.join(PKG, "_fa_torch.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_ext(force: bool, verbose: bool) -> None:
    import sysconfig

    try:
        import torch
    except ImportError as e:
        print(f"{os.path.basename(EXT)} (the binding's norm + rotation and paged calls) is not built: no torch here ({e})",
              file=sys.stderr)
        return
    base = os.path.dirname(torch.__file__)
    if not force and not _stale(EXT, [EXT_SRC, os.path.join(INCLUDE, "fa.h"), torch.__file__]):
        return
    # nvcc, for its host compiler and CUDA's headers (the one in CXX may come with another C++ runtime)
    cmd = [nvcc(), "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-o", EXT, EXT_SRC, "-I" + INCLUDE,
           *("-I" + os.path.join(base, "include", *d) for d in ((), ("torch", "csrc", "api", "include"))),
           "-I" + sysconfig.get_paths()["include"], f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"compilation failed: {' '.join(cmd)}")


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False, debug: bool = False) -> str:
    bdir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    flags = FLAGS + (["-DFA_DEBUG"] if debug else [])
    os.makedirs(bdir, exist_ok=True)
    cc = nvcc()
    headers = _headers()
    objs = []
    jobs = []
    for src in _sources():
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
            if ptxas_v:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        for cmd, r in ex.map(run, jobs):
            if r.returncode != 0 or verbose or ptxas_v:
                sys.stdout.write(r.stdout)
                sys.stderr.write(r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if force or jobs or _stale(lib, objs):
        cmd = [cc, *ARCH, "-shared", "-o", lib, *objs, "-Xcompiler", "-fPIC"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
    if not debug:
        _build_ext(force, verbose)
    return lib


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/smem usage")
    ap.add_argument("--debug", action="store_true", help="build libfa_debug.so only")
    ap.add_argument("--all", action="store_true", help="build libfa.so and libfa_debug.so")
    args = ap.parse_args()
    if args.all or not args.debug:
        print(build(force=args.force, verbose=args.verbose, ptxas_v=args.ptxas_v))
    if args.all or args.debug:
        print(build(force=args.force, verbose=args.verbose, ptxas_v=args.ptxas_v, debug=True))


if __name__ == "__main__":
    main()

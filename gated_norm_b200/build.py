"""Build libgnorm.so in-tree with nvcc for sm_100a, and the binding's module _marshal.so.

    python gated_norm_b200/build.py [--force] [--verbose]

(run it as a script: importing the package loads the library, which this script makes)

Each source is compiled to an object under ``<repo>/_build/`` (in parallel), then linked
into ``gated_norm_b200/libgnorm.so``.  The CUDA runtime is linked statically and its
symbols are kept out of the library's export table, so only the ``gnorm_*`` C entry
points are visible.  A source is recompiled when it, or any header, is newer than its
object.  _marshal.so (csrc/binding.cpp, g++ against torch's headers) is linked to libgnorm.so
beside it.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgnorm.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
SOURCES = ["api.cu", "fwd.cu", "bwd.cu", "plan.cpp", "noalloc.cu", "host_step.cu",
           "block.cu", "delta.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgnorm")


def _headers() -> list:
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(obj: str, src: str, newest_header: float) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return os.path.getmtime(src) > t or newest_header > t


def _compile(src: str, obj: str, verbose: bool) -> str:
    cmd = [nvcc(), "-c", src, "-o", obj, "-O3", "-std=c++17", "-lineinfo", *ARCH,
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose and src.endswith(".cu"):
        cmd += ["-Xptxas", "-v"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{res.stdout}\n{res.stderr}")
    return res.stdout + res.stderr


def _build_marshal() -> None:
    """Compile binding.cpp into the Python module; its only project header is gnorm.h."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    out = sysconfig.get_paths()
    src = os.path.join(CSRC, "binding.cpp")
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-shared", "-fPIC", "-O2", "-std=c++17", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-DTORCH_EXTENSION_NAME=_marshal", src, "-o", tmp, "-I", INCLUDE,
           "-I", out["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    for inc in cpp_extension.include_paths():
        cmd += ["-isystem", inc]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd += [f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python",
            f"-Wl,-rpath,{lib}", f"-L{PKG}", "-l:libgnorm.so", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, MARSHAL)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libgnorm.so and the binding's module; returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    newest_header = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    jobs = []
    objs = []
    for name in SOURCES:
        src = os.path.join(CSRC, name)
        obj = os.path.join(BUILD_DIR, name + ".o")
        objs.append(obj)
        if force or _stale(obj, src, newest_header):
            jobs.append((src, obj))
    logs = []
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = [ex.submit(_compile, s, o, verbose) for s, o in jobs]
            for f in futs:
                logs.append(f.result())
    if jobs or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), "-shared", "-o", tmp, *objs, *ARCH, "-cudart", "static",
               "-Xlinker", "--exclude-libs,ALL", "-lrt", "-lpthread", "-ldl"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)
    if force or _stale(MARSHAL, os.path.join(CSRC, "binding.cpp"),
                       os.path.getmtime(os.path.join(INCLUDE, "gnorm.h"))):
        _build_marshal()
    if verbose:
        for log in logs:
            if log.strip():
                print(log)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    args = ap.parse_args(argv)
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())

"""Builds libfox.so in place from csrc/*.cu for sm_103a with nvcc, and the binding's
_foxcall.so from csrc/fox_call.c with the C compiler (left out where Python's headers are missing: the binding
then calls by ctypes).

Each translation unit is compiled in parallel; the runtime is linked
statically so the library only needs the NVIDIA driver at load time.
Run as `python -m forget_gated_softmax_gb300.build` or call build().
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfox.so")
CALL = os.path.join(PKG, "_foxcall.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfox.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(ROOT, "include", "fox.h")
    ]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_call() -> None:
    src = os.path.join(CSRC, "fox_call.c")
    if not _stale(CALL, [src, os.path.join(ROOT, "include", "fox.h")]):
        return
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    if not cc or not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if os.path.exists(CALL):  # of an older source
            os.remove(CALL)
        print("_foxcall.so is not built (no C compiler or no Python.h): its calls go by ctypes", file=sys.stderr)
        return
    cmd = [cc, "-O2", "-std=c11", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"], src, "-o", CALL]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build of _foxcall.so failed:\n{r.stdout}{r.stderr}")


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and link libfox.so, and _foxcall.so; returns the former's path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    hdrs = _headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    jobs = [(s, o) for s, o in zip(srcs, objs) if _stale(o, [s] + hdrs)]

    def compile_one(job):
        src, obj = job
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r.returncode, r.stdout + r.stderr

    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for src, rc, out in ex.map(compile_one, jobs):
                if verbose and out.strip():
                    print(out, file=sys.stderr)
                if rc != 0:
                    raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{out}")
    if jobs or _stale(LIB, objs):
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of libfox.so failed:\n{r.stdout}{r.stderr}")
    _build_call()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))

"""Builds the CUDA libraries (sm_100a) in-tree with nvcc.

Both are plain C ABI: liblapsum_topk.so (include/lapsum_topk.h; bound in
__init__.py) from csrc/, and liblapsum_experts.so (include/lapsum_experts.h;
bound in experts.py) from csrc_experts/, each loaded with ctypes.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblapsum_topk.so")
CSRC_EXPERTS = os.path.join(PKG, "csrc_experts")
LIB_EXPERTS = os.path.join(PKG, "liblapsum_experts.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "--ftz=true",
    # a host-only function called from device code is an error, not a warning
    # (the warning leaves a kernel that does nothing)
    "--diag-error", "20011,20013,20014",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-I", INCLUDE, "-I", CSRC,
]


# the launch counter and tracer of csrc/, under this library's names
_EXPERTS_TRACE = ["-Dlapsum_%s=lapsum_experts_%s" % (n, n) for n in ("launch_count", "trace_enable", "trace_collect")]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def sources_experts():
    return sorted(glob.glob(os.path.join(CSRC_EXPERTS, "*.cu"))) + [os.path.join(CSRC, "trace.cu")]


def _headers(folder):
    return sorted(glob.glob(os.path.join(folder, "*.cuh"))) + sorted(glob.glob(os.path.join(folder, "*.h")))


def deps():
    return sources() + _headers(CSRC) + [os.path.join(INCLUDE, "lapsum_topk.h")]


def deps_experts():
    return sources_experts() + _headers(CSRC_EXPERTS) + _headers(CSRC) + _headers(INCLUDE)


def _older(out, files) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in files)


def stale(out: str = LIB) -> bool:
    return _older(out, deps())


def stale_experts(out: str = LIB_EXPERTS) -> bool:
    return _older(out, deps_experts())


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _compile(srcs, objdir, out, extra, verbose) -> str:
    os.makedirs(objdir, exist_ok=True)
    procs, objs = [], []
    for src in srcs:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [nvcc(), *NVCC_FLAGS, *(extra or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        outp, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, outp.decode(errors="replace")))
        elif verbose and outp:
            print(outp.decode(errors="replace"), file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(f"--- {s}\n{o}" for s, o in failed))
    tmp = out + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-cudart", "static",
                    "-o", tmp, *objs], check=True)
    os.replace(tmp, out)
    return out


def build(force: bool = False, out: str = LIB, extra: list[str] | None = None, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into one shared library (parallel objects)."""
    if not force and not stale(out):
        return out
    return _compile(sources(), os.path.join(PKG, "_build"), out, extra, verbose)


def build_experts(force: bool = False, out: str = LIB_EXPERTS, extra: list[str] | None = None,
                  verbose: bool = False) -> str:
    """The same for csrc_experts/ and the tracer."""
    if not force and not stale_experts(out):
        return out
    return _compile(sources_experts(), os.path.join(PKG, "_build", "experts"), out,
                    ["-I", CSRC_EXPERTS, *_EXPERTS_TRACE, *(extra or [])], verbose)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_experts(force="--force" in sys.argv, verbose="-v" in sys.argv))

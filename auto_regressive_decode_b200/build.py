"""Build libmk.so (the decode megakernel and its C ABI) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmk.so")
SOURCES = ["mk_kernel.cu", "mk_api.cu", "mk_plan.cpp", "mk_noalloc.cu", "mk_tmap.cu"]
HEADERS = ["mk_internal.h", "mk_device.h"]
# the operators around the decode step: cache append, attention over a shared prefix, token scores
OPS = os.path.join(HERE, "csrc_ops")
OPS_SOURCES = ["mk_cache.cu", "mk_append.cu", "mk_attend.cu", "mk_attend_tc.cu", "mk_score.cu"]
OPS_HEADERS = ["mk_attend.h", "mk_cache.h", "mk_ptx.h"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-Xcompiler", "-fPIC",
         "-shared", "-cudart", "static"]


def _inputs():
    root = os.path.dirname(HERE)
    return [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(OPS, f) for f in OPS_SOURCES + OPS_HEADERS] + \
        [os.path.join(root, "include", "mk.h")]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *FLAGS, *(["-Xptxas", "-v"] if verbose else []), "-o", tmp,
           *[os.path.join(CSRC, f) for f in SOURCES], *[os.path.join(OPS, f) for f in OPS_SOURCES]]
    subprocess.check_call(cmd, cwd=CSRC)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

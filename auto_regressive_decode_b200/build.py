"""Build libmk.so (the kernels and their C ABI, nvcc for sm_100a) and _mk_torch.so (the operators' torch binding) in-tree.

The binding is built where torch is installed; the C ABI does not need it."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmk.so")
SOURCES = ["mk_kernel.cu", "mk_api.cu", "mk_plan.cpp", "mk_noalloc.cu", "mk_tmap.cu"]
HEADERS = ["mk_internal.h", "mk_device.h"]
# the operators around the decode step: cache append, attention over a shared prefix, token scores
OPS = os.path.join(HERE, "csrc_ops")
OPS_SOURCES = ["mk_cache.cu", "mk_append.cu", "mk_attend.cu", "mk_attend_tc.cu", "mk_score.cu"]
OPS_HEADERS = ["mk_attend.h", "mk_cache.h", "mk_ptx.h"]
BIND = os.path.join(HERE, "_mk_torch.so")
BIND_SOURCE = os.path.join(OPS, "mk_torch.cpp")
BIND_FOR = BIND + ".for"  # the torch and the Python that it was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-Xcompiler", "-fPIC",
         "-shared", "-cudart", "static"]


def _inputs():
    root = os.path.dirname(HERE)
    return [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(OPS, f) for f in OPS_SOURCES + OPS_HEADERS] + \
        [os.path.join(root, "include", "mk.h")]


def _older(target, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in inputs)


def stale() -> bool:
    return _older(LIB, _inputs())


def _run_into(target, cmd):
    """Run `cmd` with an -o file beside the target, then put it in the target's place."""
    tmp = target + f".tmp{os.getpid()}"
    subprocess.check_call([*cmd, "-o", tmp], cwd=CSRC)
    os.replace(tmp, target)


def binding_stale() -> bool:
    """Whether the binding is older than its sources, or was built for another torch or Python."""
    root = os.path.dirname(HERE)
    if _older(BIND, [BIND_SOURCE, os.path.join(OPS, "mk_cache.h"), os.path.join(root, "include", "mk.h")]):
        return True
    try:
        with open(BIND_FOR) as f:
            return f.read() != _built_for()
    except OSError:
        return True


def _built_for() -> str:
    return f"torch {importlib.metadata.version('torch')}, Python {sys.version.split()[0]}\n"


def build_binding(force: bool = False) -> str | None:
    """The operators' torch binding: plain C++ against torch's headers, linked with libmk.so beside it.  None without torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    if not force and not binding_stale():
        return BIND
    import torch
    root = os.path.dirname(HERE)
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    lib = os.path.join(base, "lib")
    _run_into(BIND, [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", BIND_SOURCE, *[f"-I{d}" for d in inc],
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-L{HERE}", "-l:libmk.so", f"-L{lib}",
                     "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"])
    with open(BIND_FOR, "w") as f:
        f.write(_built_for())
    return BIND


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale():
        _run_into(LIB, [NVCC, *FLAGS, *(["-Xptxas", "-v"] if verbose else []), *[os.path.join(CSRC, f) for f in SOURCES],
                        *[os.path.join(OPS, f) for f in OPS_SOURCES]])
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

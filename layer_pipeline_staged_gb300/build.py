"""Build the C-ABI library ``liblps.so`` in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled in parallel, then linked into one
shared library (static CUDA runtime, no libtorch); with them the torch wrappers'
argument marshalling as a Python extension beside it (gcc, no torch headers;
its name carries the Python it is for, and it is left out, with a word on
stderr, where that Python has no headers) and what makes it quicker for one
torch (g++, that torch's headers; left out where there are none or it does not compile). Run as a module or call ``build()``;
the results sit next to this file and are git-ignored.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblps.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.c")
# Python extension: the torch wrappers' argument marshalling
MARSHAL = os.path.join(HERE, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
# and the part of it that goes through torch's C++ interface, for one version of torch
TENSORS_SRC = os.path.join(CSRC, "tensors.cpp")
TENSORS = os.path.join(HERE, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["runtime.cu", "gemv.cu", "attention.cu", "embed.cu", "noalloc.cu", "skinny.cu", "solver.cu", "stage.cu", "tcgemm.cu", "prefill.cu",
           "cache_ops.cu", "cache_rows.cu", "tile_attn.cu",
           "page_ops.cu", "paged_attn.cu", "rotary.cu", "page_evict.cu", "logits.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build liblps.so")


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_version_h(torch: str) -> str:
    return os.path.join(torch, "include", "torch", "csrc", "api", "include", "torch", "version.h")


def _torch() -> str | None:
    """The folder of the torch that this Python would import, without importing it; None: it has none, or no headers."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    where = os.path.dirname(spec.origin) if spec and spec.origin else None
    return where if where and os.path.exists(_torch_version_h(where)) else None


def _headers() -> list[str]:
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    hdrs = _headers()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *hdrs]):
            jobs.append([cc, *ARCH, *FLAGS, *(extra or []), "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            raise RuntimeError("failed: " + " ".join(cmd))

    python = sysconfig.get_paths()["include"]
    here, torch = os.path.exists(os.path.join(python, "Python.h")), _torch()
    tensors = []
    if here and torch:
        include = os.path.join(torch, "include")
        if force or _stale(TENSORS, [TENSORS_SRC, os.path.join(CSRC, "tensors.h"), _torch_version_h(torch)]):
            tmp = TENSORS + f".tmp{os.getpid()}"
            tensors = [[os.environ.get("CXX") or "g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{python}", f"-isystem{include}",
                        "-isystem" + os.path.join(include, "torch", "csrc", "api", "include"), f"-I{CSRC}", TENSORS_SRC,
                        "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]]

    def run_or_leave_out(cmd):
        try:
            run(cmd)
            os.replace(cmd[-1], TENSORS)
        except (RuntimeError, OSError) as e:
            for f in (cmd[-1], TENSORS):  # an older one may not fit the marshalling
                with contextlib.suppress(FileNotFoundError):
                    os.remove(f)
            sys.stderr.write(f"{e}\nthe torch wrappers read tensors through torch's Python interface\n")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        quicker = [ex.submit(run_or_leave_out, cmd) for cmd in tensors]
        list(ex.map(run, jobs))
        for f in quicker:
            f.result()
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([cc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    with contextlib.suppress(FileNotFoundError):
        os.remove(os.path.join(HERE, "_marshal.so"))  # an untagged one, which any Python would load
    if not here:
        sys.stderr.write(f"no Python.h in {python}: the torch wrappers of the cache operators are not built\n")
    elif force or _stale(MARSHAL, [MARSHAL_SRC, os.path.join(CSRC, "tensors.h"), os.path.join(INCLUDE, "lps.h")]):
        tmp = MARSHAL + f".tmp{os.getpid()}"
        run([os.environ.get("CC") or "gcc", "-O2", "-std=gnu11", "-Wall", "-Wextra", "-Wno-cast-function-type", "-shared", "-fPIC",
             f"-I{python}", f"-I{INCLUDE}", f"-I{CSRC}", MARSHAL_SRC, f"-L{HERE}", "-l:liblps.so", "-Wl,-rpath,$ORIGIN", "-o", tmp])
        os.replace(tmp, MARSHAL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

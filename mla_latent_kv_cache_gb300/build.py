"""Build the sm_103a C-ABI library ``_lib/libmla_gb300.so`` in-tree with nvcc.

Each translation unit is compiled in parallel; the objects are linked into
one shared library with the CUDA runtime linked statically, so the library
loads next to any PyTorch build without an rpath. ``_lib/_mla_bind.so`` (host code,
g++) holds the argument checks of the Python binding's short calls; it is built
against the installed PyTorch, and again when that changes (``_lib/_mla_bind.key``
names what it was built against). Where it cannot be built the library stands
without it, and those calls say so.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "libmla_gb300.so")
BIND = os.path.join(LIBDIR, "_mla_bind.so")
BIND_KEY = os.path.join(LIBDIR, "_mla_bind.key")
SOURCES = ["api.cu", "cache_write.cu", "decode.cu", "prefill.cu", "attn_weights.cu", "evict.cu", "rope.cu", "append.cu",
           "decode_page8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


INCLUDE = os.path.join(os.path.dirname(HERE), "include")


def _flags(extra=()):
    return ARCH + ["-I", INCLUDE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   "--expt-relaxed-constexpr", *extra]


def _inputs():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "mla.h"))
    return deps


def bind_key() -> str:
    """What _mla_bind.so has to be built against: this PyTorch and this interpreter."""
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def bind_built_for() -> str:
    """What it was built against ("" where nothing says so)."""
    try:
        with open(BIND_KEY, encoding="utf-8") as f:
            return f.read().strip()
    except OSError:
        return ""


def _bind_command(out: str) -> list:
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-I", inc, "-I",
            os.path.join(inc, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), os.path.join(CSRC, "bind.cpp"), "-o", out, "-L", lib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(LIBDIR, exist_ok=True)
    newest = max(os.path.getmtime(p) for p in _inputs())

    def fresh(f):
        return not force and not ptxas_info and os.path.exists(f) and os.path.getmtime(f) >= newest

    lib, bind = fresh(LIB), fresh(BIND) and bind_built_for() == bind_key()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(LIBDIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *_flags(extra), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if bind else ex.submit(_build_bind)
        if not lib:
            cc = nvcc()
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".tmp{os.getpid()}"
            cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static", "-lpthread", "-ldl", "-lrt"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        if binding is not None:
            binding.result()
    return LIB


def _build_bind() -> None:
    tmp = BIND + f".tmp{os.getpid()}"
    try:
        r = subprocess.run(_bind_command(tmp), capture_output=True, text=True)
        why = r.stdout + r.stderr if r.returncode != 0 else None
    except Exception as e:  # no PyTorch to build against, no compiler
        why = repr(e)
    if why is not None:
        # one that is there was built from other sources or against another PyTorch
        for f in (BIND, BIND_KEY):
            if os.path.exists(f):
                os.remove(f)
        warnings.warn("mla_rope, mla_cache_append and mla_decode_fp8_page cannot be called: the checks of their "
                      f"arguments (bind.cpp) were not built:\n{why}", stacklevel=2)
        return
    os.replace(tmp, BIND)
    with open(BIND_KEY, "w", encoding="utf-8") as f:
        f.write(bind_key() + "\n")


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_info="-v" in sys.argv))

"""In-tree build of the CUDA library ``_lib/libpa_verify.so`` for sm_103a.

Each translation unit is compiled by its own nvcc process (in parallel) and
then linked into one shared library with the CUDA runtime linked statically,
so loading it needs no CUDA toolkit on the library path. Beside it, ``_lib/pa_fast-*``
is the binding's short way into the prompt-side calls (host code over torch's
headers); the binding works without it, each of those calls taking some ten
microseconds longer on the host. It is made for one torch and one Python, which
its name says: another one does not load it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "_lib")
OBJDIR = os.path.join(LIBDIR, "obj")
LIB = os.path.join(LIBDIR, "libpa_verify.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["pa_capi.cpp", "pa_split_bf16.cu", "pa_split_fp8.cu", "pa_combine.cu", "pa_kv_write.cu", "pa_verdict.cu", "pa_tc_split.cu", "pa_tc_split_d256.cu", "pa_tc_split_d64.cu", "pa_static.cu", "pa_dyn_plan.cu",
           "pa_prefill_capi.cpp", "pa_pages.cu", "pa_rope.cu", "pa_chunk.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa_verify.so")
    return cand


def fast_path() -> str:
    """Where pa_fast stands for the torch and the Python that run; "" without torch."""
    try:
        import torch
    except ImportError:
        return ""
    return os.path.join(LIBDIR, f"pa_fast-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _current(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pa_verify.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    # -fno-gnu-unique: the launchers' per-device "attribute set" flags are function-local statics of template
    # instances; as GNU-unique symbols they would be shared with any other copy of this library loaded in the
    # same process, whose kernels would then launch without their shared-memory limit raised.
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fno-gnu-unique", "-I", INCLUDE,
           "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "cu"]
    subprocess.run(cmd, check=True)
    return obj


_fast_failed = False  # tried once a process


def _compile_fast(fast: str) -> None:
    """Compiles pa_fast.cpp against the installed torch; says so and goes on when that cannot be done."""
    global _fast_failed
    try:
        import torch
        root = os.path.dirname(torch.__file__)
        cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
        inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], cuda]
        tmp = fast + f".tmp{os.getpid()}"
        subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                        *[f"-I{i}" for i in inc], os.path.join(CSRC, "pa_fast.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"),
                        "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], check=True)
        os.replace(tmp, fast)
    except Exception as e:  # the binding's Python code does the same work
        _fast_failed = True
        if os.path.exists(fast):
            os.remove(fast)
        print(f"pa_fast was not built ({e}): calls take longer on the host", file=sys.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the library, and pa_fast, if a source is newer or they are not there; returns the library's path."""
    fast = fast_path()
    want_lib, want_fast = force or not _current(LIB), bool(fast) and not _fast_failed and (force or not _current(fast))
    if not want_lib and not want_fast:
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        made = ex.submit(_compile_fast, fast) if want_fast else None
        objs = list(ex.map(_compile, SOURCES)) if want_lib else []
        if made:
            made.result()
    if want_lib:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)

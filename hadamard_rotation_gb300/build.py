"""Compile libhq.so (the CUDA kernels and the C ABI) in-tree for sm_103a, and beside it _torch_calls.so (the
products', norms' and caches' calls over torch tensors, C++).

No fast-math: the kernels rely on IEEE division, correctly rounded reciprocals and
denormal support.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, "hq.cu"), os.path.join(CSRC, "hq_int8.cu"),
           os.path.join(CSRC, "hq_gemm.cu"), os.path.join(CSRC, "hq_norm.cu"),
           os.path.join(CSRC, "hq_gemm8.cu"), os.path.join(CSRC, "hq_kv.cu"),
           os.path.join(CSRC, "hq_smem.cu"), os.path.join(CSRC, "hq_host.cu"), os.path.join(CSRC, "hq_noalloc.cu")]
DEPS = SOURCES + [os.path.join(CSRC, "hq_kernels.cuh"), os.path.join(CSRC, "hq_int8.cuh"),
                  os.path.join(CSRC, "hq_gemm.cuh"), os.path.join(CSRC, "hq_tcgen05.cuh"),
                  os.path.join(CSRC, "hq_tensor_map.h"), os.path.join(CSRC, "hq_norm.cuh"),
                  os.path.join(CSRC, "hq_gemm8.cuh"), os.path.join(CSRC, "hq_kv.cuh"),
                  os.path.join(CSRC, "hq_kv_attend.cuh"), os.path.join(CSRC, "hq_kv_prompt.cuh"),
                  os.path.join(CSRC, "hq_internal.h"),
                  os.path.join(INCLUDE, "hq.h")]
LIB = os.path.join(PKG, "libhq.so")
CALLS_SOURCE = os.path.join(CSRC, "hq_torch.cpp")
CALLS = os.path.join(PKG, "_torch_calls.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhq.so")


def nvcc_compile_command(src: str, obj: str, extra: list[str] | None = None) -> list[str]:
    return [nvcc_path(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-c",
            "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, *(extra or []), "-o", obj, src]


def nvcc_link_command(objs: list[str], out: str) -> list[str]:
    return [nvcc_path(), ARCH, "-shared", "-o", out, *objs]


def calls_built_for() -> str:
    """What _torch_calls.so is compiled for; a copy of it is kept in the file (up_to_date)."""
    import torch

    return f"hq: torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def calls_compile_command(src: str, obj: str) -> list[str]:
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c",
            f'-DHQ_BUILT_FOR="{calls_built_for()}"',
            "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"), "-o", obj, src]


def calls_link_command(obj: str, out: str) -> list[str]:
    import torch

    return [shutil.which("g++") or "g++", "-shared", "-o", out, obj, "-L", os.path.dirname(LIB), "-lhq",
            "-Wl,-rpath,$ORIGIN", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def library_up_to_date() -> bool:
    return os.path.exists(LIB) and all(os.path.getmtime(d) <= os.path.getmtime(LIB) for d in DEPS)


def calls_up_to_date() -> bool:
    if not os.path.exists(CALLS):
        return False
    t = os.path.getmtime(CALLS)
    if any(os.path.getmtime(d) > t for d in (CALLS_SOURCE, os.path.join(INCLUDE, "hq.h"))):
        return False
    with open(CALLS, "rb") as f:
        return calls_built_for().encode() + b"\0" in f.read()


def up_to_date() -> bool:
    return library_up_to_date() and calls_up_to_date()


def _failed(what: str, rc: int):
    raise subprocess.CalledProcessError(rc, what)


def build(force: bool = False, verbose: bool = False, calls: bool = True) -> str:
    """Builds what is not up to date and returns libhq.so's path.

    libhq.so needs nvcc alone.  _torch_calls.so needs g++ and the headers of Python and of a CUDA build of torch; where it
    cannot be built this raises, after libhq.so has been linked.  ``calls=False`` leaves it out (for callers from C)."""
    library = force or not library_up_to_date()
    calls = calls and (force or not calls_up_to_date())
    tag = f".tmp{os.getpid()}"
    objs = [os.path.join(CSRC, os.path.basename(src)[:-3] + tag + ".o") for src in SOURCES] if library else []
    calls_obj = os.path.join(CSRC, "hq_torch" + tag + ".o")
    extra = ["-Xptxas", "-v"] if verbose else None
    no_calls = None
    procs, calls_proc = [], None
    try:
        # one compiler per translation unit, in parallel, then a link each
        procs = [subprocess.Popen(nvcc_compile_command(src, obj, extra)) for src, obj in zip(SOURCES, objs)]
        if calls:
            try:
                calls_proc = subprocess.Popen(calls_compile_command(CALLS_SOURCE, calls_obj))
            except (ImportError, OSError) as e:
                no_calls = e
        rcs = [pr.wait() for pr in procs]
        for src, rc in zip(SOURCES, rcs):
            if rc != 0:
                _failed(f"compiling {os.path.basename(src)}", rc)
        if library:
            tmp = LIB + tag
            subprocess.run(nvcc_link_command(objs, tmp), check=True)
            os.replace(tmp, LIB)
        if no_calls:
            raise no_calls
        if calls_proc:
            if calls_proc.wait() != 0:
                _failed(f"compiling {os.path.basename(CALLS_SOURCE)} (libhq.so is built)", calls_proc.returncode)
            tmp = CALLS + tag
            subprocess.run(calls_link_command(calls_obj, tmp), check=True)
            os.replace(tmp, CALLS)
    finally:
        for pr in [*procs, *([calls_proc] if calls_proc else [])]:
            pr.wait()
        for obj in [*objs, calls_obj]:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True, calls="--library" not in sys.argv[1:]))

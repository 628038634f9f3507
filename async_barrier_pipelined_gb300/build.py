"""Build the gemm_f16 shared library in-tree with nvcc for sm_103a.

Output: async_barrier_pipelined_gb300/_lib/libgemm_f16.so (git-ignored).
Five translation units (plan and shared host code; the kernels and entry
points of the GEMM, the attention, the paged-cache maps with rotary
positions, and the attention over a paged cache) are compiled in parallel
with one -gencode each and linked into one library, so a build takes seconds
on either the x86 build host or the aarch64 GPU host.

Beside it, _lib/paged_torch_calls.so: the paged-cache calls for torch tensors
(csrc/torch_calls.cpp, host code only, compiled against the installed torch,
and again when another torch or Python is installed).  Without torch the
library alone is built: its C ABI needs none.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG_DIR, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libgemm_f16.so")

SOURCES = [os.path.join(CSRC, f) for f in ("plan.cu", "gemm_f16.cu", "attn_f16.cu",
                                             "paged_f16.cu", "paged_attn.cu")]
HEADERS = [os.path.join(CSRC, f) for f in ("host.h", "ptx.cuh", "schedule.h", "common.cuh",
                                            "gemm_pair.cuh", "gemm_quad.cuh", "attn_f16.cuh",
                                            "attn_pair.cuh", "paged_schedule.h",
                                            "paged_small.cuh", "paged_large.cuh")]
DEPENDS = SOURCES + HEADERS + [os.path.join(INCLUDE, "gemm_f16.h"),
                               os.path.join(INCLUDE, "attn_f16.h")]

CALLS_NAME = "paged_torch_calls"
CALLS_PATH = os.path.join(LIB_DIR, CALLS_NAME + ".so")
CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")
CALLS_STAMP = os.path.join(LIB_DIR, CALLS_NAME + ".for")   # the torch that they were built for

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _compile_cmds(objs: list[str], verbose: bool) -> list[list[str]]:
    cmds = []
    for src, obj in zip(SOURCES, objs):
        cmd = [nvcc_path(), *ARCH_FLAGS, "-O3", "-std=c++17", "-lineinfo",
               "-Xcompiler", "-fPIC", "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        cmds.append(cmd)
    return cmds


def _fresh(path: str, depends: list[str]) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path)
                                        for f in depends)


def _torch_stamp() -> str | None:
    """What the torch calls are compiled against (found without importing
    torch), or None where torch is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return f"torch {version} at {spec.origin}, Python {sys.version}\n"


def _calls_fresh(stamp: str) -> bool:
    if not _fresh(CALLS_PATH, [CALLS_SOURCE, os.path.join(INCLUDE, "attn_f16.h"),
                               os.path.join(INCLUDE, "gemm_f16.h")]):
        return False
    try:
        with open(CALLS_STAMP) as f:
            return f.read() == stamp
    except OSError:
        return False


def _calls_cmd(obj: str) -> list[str]:
    from torch.utils import cpp_extension as ext
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    includes = [*ext.include_paths(), os.path.join(cuda, "include"),
                sysconfig.get_paths()["include"], INCLUDE]
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-DTORCH_EXTENSION_NAME={CALLS_NAME}",
            "-DTORCH_API_INCLUDE_EXTENSION_H", *[x for i in includes for x in ("-isystem", i)],
            "-c", CALLS_SOURCE, "-o", obj]


def _link_calls(obj: str, out: str) -> None:
    from torch.utils import cpp_extension as ext
    dirs = ext.library_paths()
    subprocess.run(["g++", "-shared", obj, "-o", out, *[f"-L{d}" for d in dirs], "-L", LIB_DIR,
                    "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python",
                    "-l:" + os.path.basename(LIB_PATH), "-Wl,-rpath,$ORIGIN",
                    *[f"-Wl,-rpath,{d}" for d in dirs]], check=True)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is older than its sources; return the library's path."""
    os.makedirs(LIB_DIR, exist_ok=True)
    calls = None
    calls_obj = os.path.join(LIB_DIR, f"{CALLS_NAME}.tmp{os.getpid()}.o")
    stamp = _torch_stamp()
    if stamp is not None and (force or not _calls_fresh(stamp)):
        calls = subprocess.Popen(_calls_cmd(calls_obj))     # beside the library's units
    try:
        _build_library(force, verbose)
        if calls is not None:
            if calls.wait():
                raise subprocess.CalledProcessError(calls.returncode, "g++ " + CALLS_SOURCE)
            tmp = CALLS_PATH + f".tmp{os.getpid()}"
            _link_calls(calls_obj, tmp)
            os.replace(tmp, CALLS_PATH)
            with open(CALLS_STAMP + f".tmp{os.getpid()}", "w") as f:
                f.write(stamp)
            os.replace(f.name, CALLS_STAMP)
    finally:
        if calls is not None:
            if calls.poll() is None:
                calls.kill()
                calls.wait()
            if os.path.exists(calls_obj):
                os.remove(calls_obj)
    return LIB_PATH


def _build_library(force: bool, verbose: bool) -> str:
    if not force and os.path.exists(LIB_PATH):
        if _fresh(LIB_PATH, DEPENDS):
            return LIB_PATH
    tag = f".tmp{os.getpid()}"
    objs = [os.path.join(LIB_DIR, os.path.basename(s)[:-3] + tag + ".o") for s in SOURCES]
    try:
        procs = [subprocess.Popen(c) for c in _compile_cmds(objs, verbose)]
        codes = [p.wait() for p in procs]
        if any(codes):
            raise subprocess.CalledProcessError(next(c for c in codes if c), "nvcc -c")
        tmp = LIB_PATH + tag
        subprocess.run([nvcc_path(), *ARCH_FLAGS, "-shared", *objs, "-o", tmp], check=True)
        os.replace(tmp, LIB_PATH)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))

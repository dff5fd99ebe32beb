"""Builds the CUDA libraries in-tree for sm_103a.

``libhstu_attn.so`` is the release build. ``libhstu_attn_checked.so`` is the
same sources compiled with ``HSTU_CHECKED``: its kernels validate every
work-list entry before using it (a debugging aid, results bit-identical).
Every translation unit of both is compiled by nvcc in one parallel pool, then
each set is linked into one shared library next to this file (the CUDA
runtime is linked statically). ``_serving.so`` is the CPython extension of the
serving and layer calls, compiled beside them against the installed torch; the libraries
need neither torch nor Python's headers, and are built where it cannot be. A
library newer than every source is not rebuilt, the extension only while torch
and Python are those it was compiled against.
"""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libhstu_attn.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
CHECKED_LIB_PATH = os.path.join(PKG, "libhstu_attn_checked.so")
EXT_SOURCE = "serving_ext.cpp"
EXT_PATH = os.path.join(PKG, "_serving.so")
EXT_STAMP = os.path.join(BUILD_DIR, "serving_built_against.txt")
# variant -> (library, object directory, extra nvcc flags)
VARIANTS = {
    "release": (LIB_PATH, BUILD_DIR, []),
    "checked": (CHECKED_LIB_PATH, os.path.join(BUILD_DIR, "checked"), ["-DHSTU_CHECKED"]),
}
SOURCES = ["plan.cu", "attn_fwd_bf16.cu", "attn_fwd_f16.cu", "attn_bwd_bf16.cu", "attn_bwd_f16.cu", "targets_only.cu", "api.cu", "noalloc.cu", "selftest.cu", "func_build.cu", "project.cu",
           "rope.cu", "cache.cu", "paged.cu", "paged_bf16.cu", "paged_f16.cu", "paged_bf16_e4m3.cu",
           "paged_f16_e4m3.cu", "embed.cu", "norm.cu", "linear.cu", "linear_bf16.cu", "linear_f16.cu", "shard.cpp"]
# Sources without HSTU_CHECKED code: the checked library links the release's
# objects of them.
SHARED = {"rope.cu", "cache.cu", "paged.cu", "paged_bf16.cu", "paged_f16.cu", "paged_bf16_e4m3.cu",
          "paged_f16_e4m3.cu", "embed.cu", "norm.cu", "linear.cu", "linear_bf16.cu", "linear_f16.cu"}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda_home, "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return found


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "hstu_attn.h"))
    return files


def up_to_date(lib: str = LIB_PATH) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _extension_against() -> str:
    """What the extension's binary depends on besides its sources."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "none"
    return f"torch {version}, python {sys.version}"


def extension_up_to_date() -> bool:
    if not up_to_date(EXT_PATH) or not os.path.exists(EXT_STAMP):
        return False
    with open(EXT_STAMP) as f:
        return f.read() == _extension_against()


def _build_extension() -> None:
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    include = os.path.join(torch_dir, "include")
    tmp = EXT_PATH + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, EXT_SOURCE), "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT_PATH)
    os.makedirs(os.path.dirname(EXT_STAMP), exist_ok=True)
    with open(EXT_STAMP, "w") as f:
        f.write(_extension_against())


def build(force: bool = False, verbose: bool = False, variants=("release", "checked")) -> str:
    """Builds the requested variants; returns the release library's path. Where
    the extension cannot be built there is a warning and none is left, so that
    the serving calls of binding.py raise; everything else is whole."""
    todo = [v for v in variants if force or not up_to_date(VARIANTS[v][0])]
    extension = force or not extension_up_to_date()
    if not todo and not extension:
        return LIB_PATH
    nvcc = _nvcc()

    def compile_one(job):
        variant, src = job
        _, obj_dir, extra = VARIANTS[variant]
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src} ({variant}):\n{r.stdout}\n{r.stderr}")
        return obj

    job_of = lambda v, src: ("release" if src in SHARED else v, src)
    jobs = sorted({job_of(v, src) for v in todo for src in SOURCES})
    for v, _ in jobs:
        os.makedirs(VARIANTS[v][1], exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(jobs), max(os.cpu_count() or 1, len(SOURCES))) + 1) as ex:
        ext = ex.submit(_build_extension) if extension else None
        objs = dict(zip(jobs, ex.map(compile_one, jobs)))
        failed = None if ext is None else ext.exception()
    for v in todo:
        lib = VARIANTS[v][0]
        tmp = lib + ".tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[objs[job_of(v, src)] for src in SOURCES]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed ({v}):\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if failed is not None:
        if os.path.exists(EXT_PATH):  # an older one, of other sources or another torch
            os.remove(EXT_PATH)
        warnings.warn(f"{os.path.basename(EXT_PATH)} has not been built: {failed}", RuntimeWarning, stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))

"""Build ``libattn_sm103a.so`` (the C-ABI attention library) in-tree with nvcc.

One ``-gencode arch=compute_103a,code=sm_103a`` target; the translation
units compile in parallel, then link into a shared library next to this file.
The CUDA runtime is linked statically, so the library does not depend on the
runtime version that PyTorch ships.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libattn_sm103a.so")
SOURCES = ["attn_api.cu", "attn_fwd_d64.cu", "attn_fwd_d128.cu", "attn_fwd_dmix.cu", "attn_fwd_alibi.cu",
           "attn_bwd_d64.cu", "attn_bwd_d128.cu", "attn_bwd_alibi.cu", "attn_bwd_dmix.cu", "attn_decode.cu", "attn_proj.cu",
           "attn_cache_q4.cu", "attn_decode_q4.cu", "attn_fwd_shared.cu", "attn_fwd_shared_alibi.cu"]
HEADERS = ["attn_internal.h", "attn_softmax.cuh", "attn_kernel_dp.cuh", "attn_kernel_bwd.cuh", "attn_kernel_bwd128.cuh", "attn_kernel_decode.cuh",
           "attn_kernel_proj.cuh", "attn_cache_q4.cuh", "attn_kernel_decode_q4.cuh", "sm103a.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(os.path.dirname(PKG), "include", "attn.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if stale) and return the path of the shared library."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    inc = ["-I", CSRC, "-I", os.path.join(os.path.dirname(PKG), "include")]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, *inc, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = f"{LIB}.{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

"""Builds libkvx.so in-tree with nvcc for sm_103a (compute_103a / sm_103a).

Translation units compile in parallel into ``_build/`` at the repository root;
the shared library lands next to this file. No CMake, no torch extension
machinery: the library is plain C ABI over the CUDA runtime (linked statically).
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libkvx.so")
SOURCES = ["plan.cpp", "abi.cpp", "attn_mma.cu", "attn_simt.cu", "gather.cu", "select.cu",
           "frame.cu", "cache.cpp", "tables.cu", "rows.cu", "tree_simt.cu",
           "tree_mma.cu", "tree_merge.cu", "window_simt.cu", "window_bf16.cu", "window_q4.cu", "window_weigh.cu", "evict.cu",
           "q4_rows.cu"]
HEADERS = [os.path.join(CSRC, "kvx_internal.h"), os.path.join(CSRC, "ptx.cuh"),
           os.path.join(CSRC, "split_merge.cuh"), os.path.join(CSRC, "tree.h"),
           os.path.join(CSRC, "tree_split.cuh"), os.path.join(CSRC, "tcgen05.cuh"),
           os.path.join(CSRC, "window.h"), os.path.join(CSRC, "window_split.cuh"),
           os.path.join(CSRC, "window_mma.cuh"),
           os.path.join(ROOT, "include", "kvx.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + HEADERS + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I", os.path.join(ROOT, "include")] + (extra or [])
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc(), "-c", os.path.join(CSRC, src), "-o", obj] + common
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))

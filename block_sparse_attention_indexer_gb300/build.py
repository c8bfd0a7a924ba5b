"""Builds libmsa.so (the C-ABI library) in-tree for sm_103a with nvcc.

Each .cu file compiles in parallel to an object under _build/, then one nvcc link makes
block_sparse_attention_indexer_gb300/libmsa.so.  Objects are rebuilt when their source or
any header changed.  Usage: python block_sparse_attention_indexer_gb300/build.py [-v] [-f]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmsa.so")
SOURCES = ["api.cu", "quant.cu", "indexer.cu", "prefill.cu", "select.cu", "attention.cu", "prefill_attn.cu", "spec_indexer.cu", "noalloc.cu",
           "api_fp8.cu", "fp8_append.cu", "fp8_attn.cu", "fp8_stream.cu",
           "fp8_tile.cu", "evict.cu", "api_prompt.cu", "prompt_attn.cu", "api_pages.cu", "pages.cu"]
HEADERS = ["msa_device.cuh", "msa_kernels.h", "api_internal.h", "select_row.cuh", "umma.cuh", "indexer_tile.cuh",
           "attention_tile.cuh", "attention_team.cuh", "fp8_device.cuh", "fp8_kernels.h", "fp8_merge.cuh",
           "prompt.h", "pages.h", "tile_split.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    env = os.environ.get("NVCC")
    if env:
        return env
    found = shutil.which("nvcc")
    if found:
        return found
    return "/usr/local/cuda/bin/nvcc"


def _newest(paths):
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    deps = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "msa.h")]
    hdr_time = _newest(deps)
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(path), hdr_time):
            return obj, ""
        cmd = [nvcc()] + FLAGS + extra + ["-c", path, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        return obj, res.stdout + res.stderr

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            if log:
                print(log)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest(objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "shared", "-o", LIB] + objs
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return LIB


if __name__ == "__main__":
    print(build(force="-f" in sys.argv, verbose="-v" in sys.argv))

"""Compile libspecverify.so (sm_103a) in-tree with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", f) for f in ("specverify.cu", "kvcache.cu", "tree.cu",
                                              "attention.cu", "attn_bf16.cu", "attn_f16.cu",
                                              "attn8_bf16.cu", "attn8_f16.cu", "rope.cu", "kv8.cu")]
INCLUDED = [os.path.join(PKG, "csrc", f) for f in ("attention.cuh", "rope.cuh")]
HEADERS = [os.path.join(ROOT, "include", f) for f in ("specverify.h", "svkv.h", "svtree.h",
                                                     "svattn.h", "svrope.h", "svkv8.h")]
OUT_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libspecverify.so")

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libspecverify.so")


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in (*SRCS, *INCLUDED, *HEADERS, __file__))


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and not extra_flags and up_to_date():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    base = [_nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include")]
    objs = [f"{tmp}.{i}.o" for i in range(len(SRCS))]

    def run(cmd: list[str]) -> None:
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    try:
        with ThreadPoolExecutor(len(SRCS)) as pool:  # one compiler process per source
            list(pool.map(run, [[*base, "-c", s, "-o", o] for s, o in zip(SRCS, objs)]))
        run([*base, "-shared", *objs, "-o", tmp])
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH

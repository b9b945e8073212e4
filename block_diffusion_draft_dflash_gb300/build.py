"""Builds the CUDA library (libdflash.so) in-tree for sm_103a with nvcc.

Translation units are compiled in parallel and linked into one shared library under
``_build/`` (``_build_checked/`` with DFLASH_CHECKED=1: device-side index checks on).  The
build is skipped when the library is newer than every source.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
# DFLASH_CHECKED=1: the checked build (device-side index checks that record DF_ERR_BOUNDS),
# kept apart from the default library
CHECKED = os.environ.get("DFLASH_CHECKED", "0") not in ("", "0")
OUT_DIR = os.path.join(PKG, "_build_checked" if CHECKED else "_build")
LIB = os.path.join(OUT_DIR, "libdflash.so")

SOURCES = ["api.cu", "gemm.cu", "attention.cu", "layers.cu", "ddtree.cu", "ddtree_static.cu", "accept.cu", "trace.cu",
           "runtime.cu", "plant.cu", "moe.cu", "kv4.cu", "kv4_attention.cu", "kv4_attention_tc.cu", "kv4_weights.cu",
           "kv4_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "dflash.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        checked = ["-DDFLASH_CHECKED=1"] if CHECKED else []
        cmd = [nvcc, *ARCH, *FLAGS, *checked, *extra_flags, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force=True))

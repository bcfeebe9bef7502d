"""Build libkvzip.so in-tree for sm_100a with nvcc.

    python -m attention_score_reduction_b200.build [--debug]

The library is written next to this file, where the Python binding loads it.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libkvzip.so")
LIB_DEBUG = os.path.join(HERE, "libkvzip_debug.so")   # with the device bounds checks
SOURCES = ["kvzip_api.cu", "score_tc.cu", "score_simt.cu", "select.cu", "select_fused.cu", "compact.cu", "heads.cu", "decode.cu",
           "cache.cu", "cache_attention.cu", "cache_attention_tc.cu", "cache_attention_merge.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _needs_rebuild(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "kvzip.h"),
                                                               os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, debug: bool = False, verbose: bool = False) -> str:
    """Compile libkvzip.so (or, with debug=True, libkvzip_debug.so with the
    device bounds checks) unless it is newer than every source."""
    lib = LIB_DEBUG if debug else LIB
    if not force and not _needs_rebuild(lib):
        return lib
    build_dir = os.path.join(ROOT, "_build_debug" if debug else "_build")
    os.makedirs(build_dir, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I" + INCLUDE, "-I" + CSRC]
    if debug:
        common += ["-DKVZIP_DEBUG"]
    if verbose:
        common += ["-Xptxas", "-v"]
    objs = [os.path.join(build_dir, src.replace(".cu", ".o")) for src in SOURCES]

    def compile_one(src, obj):
        cmd = [nvcc()] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        return subprocess.run(cmd, capture_output=True, text=True)

    with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
        results = list(pool.map(compile_one, SOURCES, objs))
    for src, r in zip(SOURCES, results):
        if r.returncode != 0 or verbose:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}")
    tmp = lib + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs + ["-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--debug", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/smem usage")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(force=bool(a.force or a.verbose), debug=a.debug, verbose=a.verbose))

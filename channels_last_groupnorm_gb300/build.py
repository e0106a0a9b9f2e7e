"""Build ``libgnsilu.so`` in-tree with nvcc for sm_103a.

The translation units are compiled in parallel and linked into a shared
library next to this file (the CUDA runtime is linked statically).
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libgnsilu.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
SOURCES = ["gn_kernels.cu", "gn_cluster.cu", "gn_capi.cu", "gn_static.cu", "rga_kernels.cu", "upconv_kernels.cu", "attn_kernels.cu", "tc_capi.cu",
           "norm_kernels.cu", "rope_kernels.cu", "pattn_kernels.cu", "pattn_forward.cu", "pattn_split.cu", "pattn_backward.cu",
           "block_capi.cu"]
HEADERS = ["gn_internal.h", "gn_math.cuh", "gn_ptx.cuh", "tc_ptx.cuh", "tc_common.cuh", "tc_internal.h", "capi_util.h",
           "block_internal.h", "block_math.cuh", "pattn_common.cuh", "pattn_tiles.cuh"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile (if needed) and return the path of libgnsilu.so."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = list(extra_flags or [])
    deps_common = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "gnsilu.h"),
                                                             os.path.abspath(__file__)]
    procs, objs = [], []
    for src in SOURCES:
        sp = os.path.join(CSRC, src)
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [sp] + deps_common):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", sp, "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed ({' '.join(cmd)}):\n{out.decode(errors='replace')}")
        if verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if force or procs or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {r.stdout.decode(errors='replace')}")
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))

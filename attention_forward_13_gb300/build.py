"""Builds the CUDA library libattn_fwd.so in-tree (attention_forward_13_gb300/_build/).

One nvcc process per translation unit, run in parallel, for sm_103a only;
then one shared-library link.  No cmake, no torch extension machinery: the
product is a plain C-ABI shared library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libattn_fwd.so")
SOURCES = ["prefill_d128.cu", "prefill_d64.cu", "prefill_keep_d128.cu", "prefill_keep_d64.cu",
           "decode_d128.cu", "decode_d64.cu", "tree_d128.cu", "tree_d64.cu", "combine.cu",
           "api.cu", "tree_api.cu", "cache.cu", "paged_noalloc.cu"]
HEADERS = ["ptx.cuh", "common.cuh", "softmax.cuh", "launch.h", "host.h", "pages.h", "prefill_kernel.cuh",
           "decode_kernel.cuh", "tree_kernel.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(os.path.dirname(HERE), "include", "attn_fwd.h"))
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    log = os.path.join(BUILD, src.replace(".cu", ".log"))
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    with open(log, "w") as fh:
        r = subprocess.run(cmd, stdout=fh, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        with open(log) as fh:
            sys.stderr.write(fh.read())
        raise RuntimeError(f"nvcc failed on {src} (see {log})")
    return obj


def build(force: bool = False) -> str:
    """Compile and link if any source is newer than the library; return its path."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))

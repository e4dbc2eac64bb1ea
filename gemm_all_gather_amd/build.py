"""Build libag.so (the HIP library behind include/ag.h) in-tree for gfx950.

    python -m gemm_all_gather_amd.build        # or: __graft_entry__.build()

Every source is compiled by hipcc for --offload-arch=gfx950 with packed
fp32 instructions disabled, then linked into gemm_all_gather_amd/libag.so.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libag.so")
BUILD_DIR = os.path.join(ROOT, "_build")
SOURCES = ["ag_host.cpp", "ag_copy.hip", "ag_gemm.hip", "ag_util.hip", "ag_linear_host.cpp", "ag_linear.hip",
           "ag_linear_forward_f16.hip", "ag_linear_forward_bf16.hip", "ag_linear_grads_f16.hip",
           "ag_linear_grads_bf16.hip", "ag_linear_i8_f16.hip", "ag_linear_i8_bf16.hip", "ag_linear_i8.hip",
           "ag_linear_q8.hip",
           "ag_rows_host.cpp", "ag_rows.hip",
           "ag_adamw_host.cpp", "ag_adamw.hip"]
ARCH = "gfx950"

COMMON_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{INCLUDE}", f"-I{CSRC}",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [hipcc()] + COMMON_FLAGS + extra + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj


def build_library(extra_flags: list[str] | None = None, out: str = LIB, verbose: bool = False) -> str:
    """Compile every source and link libag.so; returns the library path."""
    extra = list(extra_flags or [])
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), SOURCES))
    tmp = out + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, out)
    if verbose:
        print(f"built {out}")
    return out


if __name__ == "__main__":
    build_library(sys.argv[1:], verbose=True)

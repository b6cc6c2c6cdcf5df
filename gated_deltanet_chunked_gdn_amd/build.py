"""Builds libgdn.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree.

Every translation unit is compiled separately (in parallel) and linked into
``gated_deltanet_chunked_gdn_amd/libgdn.so``.  All HIP code is built with the
packed-fp32 instructions disabled.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libgdn.so")
BUILD = os.path.join(HERE, "_build")
ARCH = os.environ.get("GDN_OFFLOAD_ARCH", "gfx950")
SOURCES = ["gdn_api.cpp", "gdn_fwd.hip", "gdn_fwd_slice.hip", "gdn_bwd.hip", "gdn_rev_slice.hip", "gdn_grad_slice.hip", "gdn_selftest.hip",
           "gdn_mixer_api.cpp", "gdn_conv.hip", "gdn_norm.hip", "gdn_scan.hip",
           "gdn_scan_mma.hip", "gdn_scan_bwd.hip", "gdn_step.hip", "gdn_linear.hip", "gdn_linear_mma.hip", "gdn_group.hip"]
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-unused-command-line-argument"]


def _hipcc() -> str:
    for c in ("/opt/rocm/bin/hipcc", "hipcc"):
        if os.path.isabs(c) and os.path.exists(c):
            return c
    return "hipcc"


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(jobs: int = 0) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 1)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build())
    sys.exit(0)

"""Build libmoe_ternary.so in-tree with hipcc for gfx950.

    python -m ternary_quantized_moe_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmoe_ternary.so")
OBJ = os.path.join(PKG, "_build")
SOURCES = ["host_codec.cpp", "moe_capi.hip", "moe_kernels.hip", "moe_experts.hip", "moe_dense.hip", "moe_quant.hip", "moe_ple.hip", "moe_mtp.hip", "moe_router_delta.hip", "moe_norm.hip", "moe_fp8_linear.hip", "moe_sample.hip", "moe_attention.hip", "moe_decode.hip", "moe_kv_cache.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    "-Wno-unused-function",
    # no packed fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln and ln.strip()]
    if res.returncode != 0:
        sys.stderr.write("\n".join(msgs) + "\n")
        raise RuntimeError(f"hipcc failed with exit code {res.returncode}: {' '.join(cmd[-3:])}")
    if msgs and verbose:
        sys.stderr.write("\n".join(msgs) + "\n")


def build(verbose: bool = True, jobs: int = 0) -> str:
    """Compile every source to an object (in parallel), then link the library."""
    from concurrent.futures import ThreadPoolExecutor
    os.makedirs(OBJ, exist_ok=True)
    compile_flags = [f for f in FLAGS if f != "-shared"]
    objs, cmds = [], []
    for s in SOURCES:
        obj = os.path.join(OBJ, os.path.splitext(s)[0] + ".o")
        objs.append(obj)
        cmds.append([HIPCC, *compile_flags, "-c", os.path.join(CSRC, s), "-o", obj])
    n = jobs or min(len(cmds), os.cpu_count() or 1, 16)
    with ThreadPoolExecutor(n) as ex:
        list(ex.map(lambda c: _run(c, verbose), cmds))
    tmp = LIB + ".tmp"
    _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build()

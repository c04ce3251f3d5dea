"""Build libconvfwd.so (host planner + gfx950 kernels) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libconvfwd.so")
# measurement probes for the benchmark (measured ceilings), a library of their own
PROBE_SRC = "probe_ceilings.hip"
PROBE_LIB = os.path.join(PKG, "libconvprobe.so")

SOURCES = ["conv_plan.cpp", "pool_plan.cpp", "conv_host.cpp", "k_pool.hip", "k_convint.hip", "k_convint_rs.hip", "k_winograd.hip", "k_igemm.hip", "k_direct.hip", "k_halo.hip", "k_rowshift.hip", "k_pointwise.hip", "k_rowband.hip", "k_grouped.hip", "k_pointwise32.hip",
           "linear_plan.cpp", "grad_clip_plan.cpp", "k_linear.hip", "k_linear_f16.hip", "k_linear_bf16.hip",
           "k_linear_f32.hip", "k_linear_stream.hip", "k_linear_grad.hip", "k_grad_clip.hip",
           "rows_plan.cpp", "linear_int8_plan.cpp", "k_linear_int8.hip", "k_layer_norm.hip",
           "k_layer_norm_grad.hip", "k_dropout.hip", "k_quantize.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    "-Wall", "-Wno-unused-function",
    # packed-fp32 instructions stay off (plain v_fma_f32 / MFMA only)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _compile(src: str) -> str:
    out = os.path.join(BUILD, os.path.basename(src) + ".o")
    lang = ["-x", "hip"]
    cmd = [HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc link failed")
    os.replace(tmp, LIB)
    probe_obj = _compile(PROBE_SRC)
    tmp = PROBE_LIB + ".tmp"
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, probe_obj],
                       capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("hipcc link failed (probe library)")
    os.replace(tmp, PROBE_LIB)
    if verbose:
        print("built", LIB, "and", PROBE_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)

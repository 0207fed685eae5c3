"""Build libmxcast.so for gfx950 in-tree with hipcc (no GPU needed)."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmxcast.so")
SOURCES = ["mx_api.hip", "mx_cast.hip", "mx_blocked.hip", "mx_rowwise.hip", "mx_tensorwise.hip", "mx_gemm.hip",
           "mx_train_api.hip", "mx_norm.hip", "mx_router.hip", "mx_gated_act.hip", "mx_wgrad.hip",
           "mx_fp4_api.hip", "mx_fp4_cast.hip", "mx_mm_gemm.hip", "mx_mm_ffn.hip", "mx_decode.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fvisibility=hidden",
    "-Wall",
    # keep the compiler from forming packed-fp32 VALU instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _hipcc(args, verbose: bool):
    cmd = [HIPCC, *FLAGS, *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed (%d):\n%s" % (res.returncode, err))
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build(verbose: bool = False) -> str:
    """Compile every source, several at a time, and link them into
    fp8_precision_quantization_amd/libmxcast.so."""
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as objs, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        pairs = [(os.path.join(CSRC, s), os.path.join(objs, s + ".o")) for s in SOURCES]
        jobs = [pool.submit(_hipcc, ["-c", "-I", INCLUDE, "-I", CSRC, src, "-o", obj], verbose) for src, obj in pairs]
        for job in jobs:
            job.result()
        _hipcc(["-shared", *(obj for _, obj in pairs), "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))

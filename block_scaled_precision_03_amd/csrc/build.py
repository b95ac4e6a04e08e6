"""Build libmxgemm.so (the HIP library) for gfx950 with hipcc.

Usage: python -m block_scaled_precision_03_amd.csrc.build   (or call build()).
Always recompiles; writes block_scaled_precision_03_amd/libmxgemm.so.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
OUT = os.path.join(PKG, "libmxgemm.so")
OBJDIR = os.path.join(ROOT, "_build")
SOURCES = ["api.hip", "k_dense_mx4.hip", "k_dense_mx5.hip", "k_dense_tw4.hip", "k_dense_tw5.hip",
           "k_dense_fp4.hip", "k_small.hip", "k_grouped.hip", "k_int8.hip", "k_moe.hip", "k_experts.hip",
           "k_residual.hip", "k_res_mx4.hip", "k_res_mx5.hip", "k_res_tw4.hip", "k_res_tw5.hip", "k_res_fp4.hip", "k_rows.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result", "-I", os.path.join(ROOT, "include"),
]


def _compile(src):
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(HERE, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr[-4000:]))
    return obj


def build(verbose=False):
    os.makedirs(OBJDIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr[-4000:])
    os.replace(tmp, OUT)
    if verbose:
        print(OUT)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

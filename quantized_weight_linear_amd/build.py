"""Build libnq.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree.

    python -m quantized_weight_linear_amd.build

Every source is compiled to an object under ``_build/`` (in parallel) and
linked into ``quantized_weight_linear_amd/libnq.so``.  Flags:
  -O3, C++17, gfx950 only;
  -ffp-contract=off: no silent a*b+c fusion, every rounding is the one the
   source writes (explicit fmaf where a fused multiply-add is meant);
  packed FP32 instructions disabled (the scalar forms are used instead).
"""

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libnq.so")

SOURCES = ["nq_abi.cpp", "nq_convert.hip", "nq_gemv.hip", "nq_gemv_fp8row.hip", "nq_gemv_mxfp8.hip",
           "nq_gemv_bf16.hip", "nq_gemv_q8g64.hip", "nq_gemv_q4g64.hip", "nq_gemv_q8g32.hip", "nq_gemv_a8.hip",
           "nq_gemv_qb.hip", "nq_gemm.hip", "nq_attn_prompt.hip", "nq_attn_tree.hip", "nq_kv_pages.hip",
           "nq_probe.hip"]

FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-unused-result", "-I", INCLUDE, "-I", CSRC]


def hipcc():
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libnq.so)")


# Per-source additions.  The GEMM, the GEMVs and attention keep their MFMA results in
# ordinary VGPRs, where the FP32 rescales read them directly (no copy out of
# AGPRs per element; measured 5-12 % faster on the grouped GEMV formats).
EXTRA = {name: ["-mllvm", "-amdgpu-mfma-vgpr-form"] for name in SOURCES if name.startswith(("nq_gemm", "nq_gemv", "nq_attn"))}


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc()] + FLAGS + EXTRA.get(src, []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if verbose and out.strip():
        print(out)
    return obj


def build(verbose=False):
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), max(1, int(os.environ.get("MAX_JOBS", os.cpu_count() or 4))))
    with ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))

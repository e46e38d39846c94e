"""Build the gfx950 HIP library libgptq_mi355x.so in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgptq_mi355x.so")
BUILD = os.path.join(HERE, "_build")

SOURCES = ["gptq_abi.cpp", "syrk_f16.hip", "chol_f64.hip", "sweep.hip", "act_order.hip", "infer.hip",
           "linear_mfma.hip", "accumulate_noalloc.hip", "adapters.hip", "gemm_f16.hip", "head.hip",
           "decode_adapters.hip", "linear_wide.hip", "train_abi.cpp"]

# Per-file code generation options.  The fp64 kernels keep their MFMA
# accumulators in ordinary VGPRs: with the default AGPR form the compiler
# copies fp64 accumulators between the two register files around every
# MFMA, which halves fp64 MFMA throughput.  (The fp16 SYRK needs the AGPRs
# for its 256 accumulator registers per lane.)
EXTRA = {"chol_f64.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
    # no packed fp32 (v_pk_fma_f32 & co.) anywhere
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
    "-Wall", "-Wno-unused-result",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src + ".o")
    cmd = [HIPCC, *FLAGS, *EXTRA.get(src, []), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        # keep warnings visible (the host pass may warn about the gfx feature flag)
        lines = [ln for ln in r.stderr.splitlines() if "packed-fp32-ops" not in ln]
        if any(ln.strip() for ln in lines):
            sys.stderr.write("\n".join(lines) + "\n")
    return obj


def build(verbose: bool = True) -> str:
    """Compile every source for gfx950 and link the shared library. Always
    recompiles (the caller asked for a build)."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(min(len(SOURCES), 8)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()

"""Build libmoe.so (HIP for gfx950) in-tree with hipcc."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
# the dense operators, apart from the MoE layer's kernels: bench.py takes counters of those as
# current for as long as csrc/ is unchanged
CSRC_DENSE = os.path.join(PKG, "csrc_dense")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")

SOURCES = ["moe_api.hip", "route.hip", "permute.hip", "ffn_skinny.hip", "ffn_mfma.hip",
           "combine.hip", "decode.hip", "pager.hip",
           "ffn_mx.hip"]
SOURCES_DENSE = ["norm_quant.hip", "linear_i8.hip", "dense_api.hip"]
ARCH = "gfx950"
FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 ops stay off (hipcc -O3 would otherwise form them from scalar code)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE fp32 division: the FP8 activation scales and codes depend on it
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Wno-unused-result",
    f"-I{INCLUDE}", f"-I{CSRC}", f"-I{CSRC_DENSE}",
]


def _hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the MoE library needs ROCm's hipcc to build")


def build(verbose: bool = False) -> str:
    """Compile every source for gfx950 and link libmoe.so.  Always rebuilds."""
    hipcc = _hipcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(path: str) -> str:
        src = os.path.basename(path)
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        cmd = [hipcc, *FLAGS, "-c", path, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{res.stderr}")
        if verbose and res.stderr.strip():
            print(res.stderr)
        return obj

    paths = ([os.path.join(CSRC, s) for s in SOURCES]
             + [os.path.join(CSRC_DENSE, s) for s in SOURCES_DENSE])
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(paths))) as ex:
        objs = list(ex.map(compile_one, paths))
    tmp = LIB + ".tmp"
    cmd = [hipcc, "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))

"""Build libgdn.so (HIP for gfx950) in place with hipcc.

    python -m gated_deltanet_chunked_gdn_amd.build

Every source is compiled for gfx950 only.  Packed-fp32 instructions are
switched off for the device code (-packed-fp32-ops); hipcc's host pass reports
that feature as unknown, which is harmless.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libgdn.so")
BUILD_DIR = os.path.join(ROOT, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["gdn_abi.cpp", "gdn_noalloc.cpp", "gdn_chunk_fwd.hip", "gdn_chunk_chain.hip", "gdn_chunk_bwd.hip", "gdn_recurrent.hip", "gdn_prologue.hip",
           "gdn_epilogue.hip", "gdn_layer_abi.cpp", "gdn_scan_split.cpp", "gdn_step.hip", "gdn_conv.hip", "gdn_scan.hip", "gdn_scan_time.hip", "gdn_scan_bwd.hip", "gdn_kda.hip", "gdn_kda_bwd.hip", "gdn_copy.hip"]
COMMON = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-Wno-unused-parameter", f"-I{INCLUDE}", f"-I{CSRC}"]


# The state pass keeps its MFMA accumulators in VGPRs: it touches them with VALU
# code between products, which AGPR accumulators would turn into copies.
EXTRA = {"gdn_chunk_chain.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(line for line in r.stderr.splitlines() if noise not in line)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{err}")
    if err.strip():
        print(err, file=sys.stderr)
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print(f"built {OUT}")
    return OUT


if __name__ == "__main__":
    build()

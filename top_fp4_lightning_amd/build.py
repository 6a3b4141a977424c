"""Build libfp4idx.so in-tree with hipcc for gfx950 (one object per source, compiled in parallel)."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCES = ["api.hip", "quantize.hip", "score.hip", "score_multi.hip", "select.hip", "mainkv.hip", "mask.hip",
           "rope.hip", "attend.hip", "distill.hip"]
OUT = os.path.join(HERE, "libfp4idx.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # keep the compiler from emitting packed fp32 VALU ops (v_pk_fma/mul/add_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # matrix-instruction results in ordinary VGPRs: the epilogue reads them without
    # v_accvgpr_read copies
    "-mllvm", "-amdgpu-mfma-vgpr-form",
]

# Scoring never meets a NaN: FP4 codes are finite, E8M0 scales stop at 2^127 (the NaN byte 255
# is never produced and is rejected by contract), weights are finite. Without NaN semantics a
# float max needs no operand canonicalisation and folds the cross-lane move into itself.
PER_FILE = {"score.hip": ["-fno-honor-nans"], "score_multi.hip": ["-fno-honor-nans"]}


def _compile(src: str, obj: str) -> None:
    name = os.path.basename(src)
    cmd = [HIPCC, *FLAGS, *PER_FILE.get(name, []), "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {name} ({res.returncode}):\n{res.stderr}")


def build_library(verbose: bool = False) -> str:
    srcs = [os.path.join(HERE, "csrc", s) for s in SOURCES]
    with tempfile.TemporaryDirectory(prefix="fp4idx_build_") as tmpdir:
        objs = [os.path.join(tmpdir, os.path.splitext(os.path.basename(s))[0] + ".o") for s in srcs]
        if verbose:
            print(" ".join([HIPCC, *FLAGS, "-c", "<src>"]), flush=True)
        with ThreadPoolExecutor(len(srcs)) as ex:
            list(ex.map(_compile, srcs, objs))
        tmp = OUT + ".tmp"
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc link failed ({res.returncode}):\n{res.stderr}")
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build_library(verbose=True))

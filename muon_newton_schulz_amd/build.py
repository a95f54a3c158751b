"""Build libmuon.so (gfx950 only) in-tree with hipcc.

    python -m muon_newton_schulz_amd.build
"""

from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmuon.so")
SOURCES = ["muon_abi.hip", "elementwise.hip", "ns_gemm.hip", "ns_f32.hip", "ns_small.hip", "guard.hip",
           "clip.hip", "embed.hip", "lm_loss.hip", "experts.hip"]
# stand-alone measurement programs: the GPU's sustained bf16 MFMA rate and
# its HBM stream rates
PROGRAMS = [("mfma_ceiling", "mfma_ceiling.hip"), ("hbm_ceiling", "hbm_ceiling.hip")]

JOBS = min(8, os.cpu_count() or 1)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # no packed-fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]


def _hipcc(cmd, out, verbose):
    tmp = out + ".tmp"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)
    os.replace(tmp, out)


def build(verbose: bool = True) -> str:
    # one object per source, compiled side by side, then one link
    compile_flags = [f for f in FLAGS if f != "-shared"]
    exe_flags = [f for f in compile_flags if f != "-fPIC"]
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(JOBS) as pool:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        jobs = [pool.submit(_hipcc, [HIPCC, *compile_flags, "-c", os.path.join(CSRC, s)], o, verbose)
                for s, o in zip(SOURCES, objs)]
        jobs += [pool.submit(_hipcc, [HIPCC, *exe_flags, os.path.join(CSRC, src)],
                             os.path.join(PKG, exe), verbose) for exe, src in PROGRAMS]
        for j in jobs:
            j.result()
        _hipcc([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objs], LIB, verbose)
    return LIB


if __name__ == "__main__":
    build()

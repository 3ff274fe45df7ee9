"""Builds libmoe_hotpath.so (gfx950) in-tree with hipcc; libmoe_ceiling.so,
the benchmark's read-stream and MFMA-rate probes (not part of the hot path's C
ABI); and libmoe_hotpath_trace.so, the same sources with the clock-stamp trace
compiled in (MOE_TRACE=1, csrc/trace.h), which `python -m
combine_expert_histogram_amd.trace` loads.

Usage: python -m combine_expert_histogram_amd.build [-v] [--no-trace]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoe_hotpath.so")
SOURCES = ["api.hip", "layout.hip", "quant.hip", "gemm1.hip", "stage2.hip", "combine.hip",
           "route_topk.hip", "few_token.hip", "dense.hip", "dense_few.hip", "dense_tile_nt.hip", "dense_tile_nn.hip",
           "dense_tile_tn.hip", "dense_tile_pair.hip", "norm.hip"]
TRACE_LIB = os.path.join(PKG, "libmoe_hotpath_trace.so")
CEILING_LIB = os.path.join(PKG, "libmoe_ceiling.so")
CEILING_SOURCES = ["ceiling.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build the HIP library)")


def flags() -> list[str]:
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
        # no fast-math: the quant's IEEE divisions must stay correctly rounded
        "-fno-fast-math", "-ffp-contract=on",
        # keep the compiler from emitting packed fp32 arithmetic
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wno-unused-command-line-argument",
        f"-I{INCLUDE}", f"-I{CSRC}",
    ]


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")


def _compile(source: str, out: str, verbose: bool, extra: tuple[str, ...] = ()) -> str:
    _run([hipcc(), *(f for f in flags() if f != "-shared"), *extra, "-c", os.path.join(CSRC, source), "-o", out], verbose)
    return out


def build(verbose: bool = False, trace: bool = True) -> str:
    libs = [(LIB, SOURCES, ()), (CEILING_LIB, CEILING_SOURCES, ())]
    if trace:
        libs.append((TRACE_LIB, SOURCES, ("-DMOE_TRACE=1",)))
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        # every source of every library by itself, the slow ones first; then one link a library
        jobs = [(os.path.join(tmp, f"{i}_{s}.o"), s, extra) for i, (_, sources, extra) in enumerate(libs) for s in sources]
        jobs.sort(key=lambda job: -os.path.getsize(os.path.join(CSRC, job[1])))
        for f in [pool.submit(_compile, s, out, verbose, extra) for out, s, extra in jobs]:
            f.result()
        for i, (lib, sources, _) in enumerate(libs):
            _run([hipcc(), *flags(), *(os.path.join(tmp, f"{i}_{s}.o") for s in sources), "-o", lib + ".tmp"], verbose)
            os.replace(lib + ".tmp", lib)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, trace="--no-trace" not in sys.argv))

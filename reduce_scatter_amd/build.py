"""Build ``libar.so`` (the HIP kernels and the C ABI) for gfx950 with hipcc.

``python reduce_scatter_amd/build.py`` (by path: it imports nothing from the
package, whose import would load the library being replaced).
Objects are compiled in parallel into ``reduce_scatter_amd/_build/`` and
linked into ``reduce_scatter_amd/libar.so``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libar.so")
SOURCES = ["tree.hip", "tree_stream.hip", "tree_reg.hip", "fused.hip", "fused_rs.hip", "ring.hip", "split.hip", "fused_phase.hip", "elem.hip", "reshard.hip",
           "logprobs.hip", "distill.hip", "norm.hip", "embed.hip", "gradnorm.hip", "api.cpp", "plan.cpp", "reshard_api.cpp", "vocab_api.cpp",
           "layer_api.cpp"]

ARCH = "gfx950"
# -ffp-contract=off: a multiply followed by an add (the avg pre-scale, then
# the hop's add) must round twice, exactly as written, never fuse into an FMA.
# The packed-fp32 feature is turned off: only scalar fp32 instructions.
FLAGS = ["-O3", "-std=c++17", "-fPIC", "-ffp-contract=off", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", os.path.join(ROOT, "include")]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain (ROCm) is required to build libar.so")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source and link libar.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp, "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)

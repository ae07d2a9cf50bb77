"""Builds libgbdt_hip.so (the C-ABI library) for gfx950 with hipcc, in-tree."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libgbdt_hip.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["gbdt_kernels.hip", "gbdt_driver.hip", "gbdt_predict.hip", "gbdt_distill.hip", "gbdt_select.hip",
           "gbdt_policy.hip", "gbdt_route.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# -ffp-contract=off: FP64 gain / weight / prediction arithmetic is evaluated
# one IEEE operation at a time, as on the CPU.  The packed-FP32 target
# feature is switched off for all device code.  Kernel arguments are
# preloaded into SGPRs at wave launch (the first 16 dwords), which saves the
# kernels' first scalar round trip; without firmware support the code object's
# own prologue loads them instead.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall", "-Wno-unused-function",
    "-I" + INCLUDE, "-I" + CSRC,
]


def build(verbose: bool = False) -> str:
    """Compiles the sources side by side, then links them."""
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as objects:
        jobs, outs = [], []
        for src in SOURCES:
            out = os.path.join(objects, src + ".o")
            cmd = [HIPCC] + [f for f in FLAGS if f != "-shared"] + ["-c", os.path.join(CSRC, src), "-o", out]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append((cmd, subprocess.Popen(cmd)))
            outs.append(out)
        for cmd, job in jobs:
            if job.wait() != 0:
                for _, other in jobs:
                    other.wait()
                raise subprocess.CalledProcessError(job.returncode, cmd)
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + outs + ["-o", tmp], check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    print(LIB_PATH)
    sys.exit(0)

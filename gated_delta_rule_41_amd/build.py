"""Build libkda.so (the HIP kernels and the C ABI) in-tree for gfx950."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")
SOURCES = ["kda_api.hip", "kda_fwd.hip", "kda_fwd16.hip", "kda_bwd.hip", "kda_decode.hip", "kda_split.hip", "kda_exact.hip", "kda_scan16.hip",
           "kda_staged.hip", "kda_linear_api.hip", "kda_linear_fwd.hip", "kda_linear_bwd.hip", "kda_linear_decode.hip", "kda_tree.hip", "kda_layer_api.hip",
           "kda_norm.hip", "kda_conv.hip", "kda_selective_states.hip", "kda_selective_fwd.hip", "kda_selective_bwd.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # Packed fp32 VALU instructions are kept out of the device code.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # a*b+c is fused only inside one source expression, so every inlined copy
    # of a step (prologue and loop bodies) rounds the same way and results do
    # not depend on where a sequence is split.
    "-ffp-contract=on",
    "-Wno-unused-result",
]


# Flags of single sources.  The kernels of the linear rule and the trees keep their accumulators
# in the same registers as everything else: with separate accumulation registers every scaling
# of a state block was a move out, a multiply and a move back.
SOURCE_FLAGS = {s: ["-mllvm", "-amdgpu-mfma-vgpr-form"]
                for s in ("kda_linear_fwd.hip", "kda_linear_bwd.hip", "kda_linear_decode.hip", "kda_tree.hip")}


def build(verbose: bool = False, extra_flags=None) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    common = [f for f in HIPCC_FLAGS if f != "-shared"] + list(extra_flags or []) + ["-I", os.path.join(ROOT, "include")]
    tmp = LIB + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("hipcc failed building libkda.so")
        if verbose:
            noise = [ln for ln in res.stderr.splitlines() if "packed-fp32-ops" not in ln and ln.strip()]
            if noise:
                print("\n".join(noise[:40]))

    with tempfile.TemporaryDirectory() as work:
        def compile_one(source):
            obj = os.path.join(work, source + ".o")
            run([hipcc] + common + SOURCE_FLAGS.get(source, []) + ["-c", os.path.join(CSRC, source), "-o", obj])
            return obj

        with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            objs = list(pool.map(compile_one, SOURCES))
        run([hipcc] + HIPCC_FLAGS + objs + ["-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))

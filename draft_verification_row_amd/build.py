"""Build the HIP library libspecverify.so for gfx950, in-tree.

    python -m draft_verification_row_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRCS = [os.path.join(CSRC, f) for f in ("spec_verify.hip", "row_ops.hip", "linear.hip", "embedding.hip",
                                           "gated.hip", "cross_entropy.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libspecverify.so")

# Packed fp32 instructions are disabled for every HIP translation unit: the
# library's float code is written for scalar v_*_f32 forms.
HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "hipcc"


def _run(cmd) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (res.stderr or "").splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if err.strip():
        print(err, file=sys.stderr)


def build_library(out: str = LIB, extra_flags=()) -> str:
    """Compiles the sources side by side and links them into `out`."""
    tmp = out + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(s) + ".o") for s in SRCS]
        with ThreadPoolExecutor(len(SRCS)) as pool:
            list(pool.map(lambda so: _run([hipcc(), *HIPCC_FLAGS, *extra_flags, "-I" + INCLUDE,
                                           "-c", "-o", so[1], so[0]]), zip(SRCS, objs)))
        _run([hipcc(), "--offload-arch=gfx950", "-shared", "-o", tmp, *objs])
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build_library())

"""What the training operators launch stays in the buffers of the call: their
sources are compiled for the host with tests/sanitize/training_launches.cpp,
which stands in for the HIP runtime, calls every entry point over sizes, types
and alignments, and compares the ranges that each launch reads and writes with
what the caller gave.  No kernel runs; no GPU is needed."""
import os

import pytest

from test_sanitizers import CLANGXX, HERE, HIPCC, ROOT, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)),
                    reason="ROCm toolchain not available")
def test_launches_stay_in_their_buffers(tmp_path):
    obj, exe = str(tmp_path / "launches.o"), str(tmp_path / "launches")
    _run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-x", "hip", "-O1", "-std=c++17",
          "-I" + os.path.join(ROOT, "include"), "-c", "-o", obj, os.path.join(HERE, "training_launches.cpp")])
    _run([CLANGXX, "-o", exe, obj])
    r = _run([exe], timeout=300)
    assert ", 0 failures" in r.stdout

"""CPU sanitizer run of the training operators' host code: embedding.hip,
gated.hip and cross_entropy.hip are compiled with AddressSanitizer and
UndefinedBehaviorSanitizer on the host pass (device code as usual for gfx950)
and driven by tests/sanitize/training_driver.cpp, which asks every size query
over the range of its arguments and calls every entry point with arguments it
must reject.  No kernel is launched; no GPU is needed."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_sanitizers import CLANGXX, ENV, HERE, HIPCC, ROOT, _run

SOURCES = ["embedding.hip", "gated.hip", "cross_entropy.hip"]


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANGXX)),
                    reason="ROCm toolchain not available")
def test_training_operators_host_code_under_asan_and_ubsan(tmp_path):
    inc = "-I" + os.path.join(ROOT, "include")
    csrc = os.path.join(ROOT, "draft_verification_row_amd", "csrc")
    sanitized = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                 "-Xarch_host", "-fno-sanitize-recover=all"]

    def compile_one(name):
        obj = str(tmp_path / (name + ".o"))
        _run([HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *sanitized, inc, "-c", "-o", obj,
              os.path.join(csrc, name)])
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    lib = str(tmp_path / "libtraining_asan.so")
    _run([HIPCC, "--offload-arch=gfx950", "-shared", *sanitized, "-o", lib, *objs])
    exe = str(tmp_path / "training_driver")
    _run([CLANGXX, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", inc,
          "-o", exe, os.path.join(HERE, "training_driver.cpp"), "-L" + str(tmp_path), "-ltraining_asan",
          "-Wl,-rpath," + str(tmp_path)])
    r = _run([exe], env=ENV, timeout=300)
    assert "0 failures" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr

"""include/q3_block.h's host code under AddressSanitizer and
UndefinedBehaviorSanitizer: tests/test_block_abi.py (refusals before any HIP
call, workspace sizes) in a child interpreter against the instrumented build, as
tests/test_abi_sanitized.py does for q3.h.  CPU only: no kernel is launched."""
import os
import subprocess
import sys

import pytest

from conftest import ROOT
from test_abi_sanitized import CHILD, _stale


def test_block_abi_suite_under_host_sanitizers():
    from bit_fp8_codebook_amd import build
    try:
        rt = build.asan_runtime()
        build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    srcs = build.sources() + [os.path.join(ROOT, "include", h) for h in ("q3.h", "q3_block.h")]
    if _stale(build.ASAN_LIB, srcs):
        build.build_asan(verbose=False)
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), lib=build.ASAN_LIB,
                        suite=os.path.join(ROOT, "tests", "test_block_abi.py"))
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", code], env=env, cwd=ROOT, capture_output=True, text=True, timeout=900)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in r.stdout

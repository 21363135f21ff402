"""Where the small products stop staging whole activations in LDS when K ends
inside a 512-column step.  Rows take K rounded up to four groups and a pad of 16
bytes, not whole steps; the split of the streamed form shows in the workspace
that the library asks for.  No GPU."""
import os

import pytest

BUDGET = 136 * 1024   # bytes of LDS for staged activations, 1 KB of them zeros


@pytest.fixture(scope="module")
def L():
    from bit_fp8_codebook_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from bit_fp8_codebook_amd import build
        build.build(verbose=False)
    return _lib.lib()


@pytest.mark.parametrize("k,last", [(2304, 29), (4864, 14), (2880, 23), (5280, 12), (4096, 16), (2048, 33)])
def test_last_staged_token_count(L, k, last):
    row = (k // 32 + 3) // 4 * 4 * 64 + 16
    assert (BUDGET - 1024) // row == last
    for m in range(1, 65):
        streamed = L.q3_gemm_small_m_workspace_bytes(1024, k, m) > 0
        assert streamed == (m > last), m

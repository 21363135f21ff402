"""The large product kernel's sums live in accumulation registers that its
assembly statements write without the compiler knowing when they are done.  That
holds as long as the compiler moves none of them inside the loop, and each step's
last product is followed at once by its wait: checked on the assembly that the
build's own flags give.  CPU only."""
import os
import re
import subprocess

import pytest


def test_no_sum_moves_between_the_products(tmp_path):
    from bit_fp8_codebook_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    src = next(s for s in build.sources() if os.path.basename(s) == "q3_gemm.hip")
    out = str(tmp_path / "gemm.s")
    subprocess.run([hipcc, *build.COMMON, *build.DEVICE_FLAGS, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   capture_output=True)
    kernels = [k for k in re.split(r"\n(?=_Z\S+:)", open(out).read()) if re.match(r"_Z\S*gemm_kernelILi8ELi8E", k)]
    assert len(kernels) == 2
    for k in kernels:
        lines = [x.strip() for x in k.split("\n")]
        products = [i for i, x in enumerate(lines) if x.startswith("v_mfma")]
        assert len(products) == 128                       # two halves of 8 x 8 in one loop body
        body = lines[products[0]:products[-1] + 1]
        assert not [x for x in body if x.startswith("v_accvgpr")]
        assert lines[products[-1] + 1:products[-1] + 3] == ["s_nop 15", "s_nop 3"]

"""The heads' kernel reads no row that belongs to no sequence of a batch: such a row
need not be there.  Seen on the assembly that the build's own flags give, in which
the search for a row's sequence (the only counting of a ballot) and its way out
stand in front of every load of a row (16 bytes a lane).  CPU only."""
import os
import re
import subprocess

import pytest


def test_the_sequence_is_found_before_a_row_is_read(tmp_path):
    from bit_fp8_codebook_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    src = next(s for s in build.sources() if os.path.basename(s) == "q3_rope.hip")
    out = str(tmp_path / "rope.s")
    subprocess.run([hipcc, *build.COMMON, *build.DEVICE_FLAGS, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   capture_output=True)
    kernels = [k for k in re.split(r"\n(?=_Z\S+:)", open(out).read()) if re.match(r"_Z\S*19qk_norm_rope_kernel", k)]
    assert len(kernels) == 15      # 5 lane counts, 3 pairings
    for k in kernels:
        lines = [x.strip() for x in k[:k.index(".section")].split("\n")]
        counts = [i for i, x in enumerate(lines) if x.startswith("s_bcnt1_i32_b64")]
        rows = [i for i, x in enumerate(lines) if re.match(r"(global|flat|buffer)_load_dwordx4", x)]
        assert counts and rows
        # the way out stands between them
        assert max(counts) < min(rows), k.split(":")[0]
        assert any(lines[i].startswith("s_cbranch") for i in range(max(counts), min(rows)))

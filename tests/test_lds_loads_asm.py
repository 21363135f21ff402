"""The attention kernels' loads to LDS set the register that holds their target by
themselves; the compiler, which uses it for such loads of its own, has to know.
Seen on the assembly of a small kernel that has one between two of the compiler's:
the second of those sets the register again.  CPU only."""
import re
import subprocess

import pytest

PROBE = r"""
#include "q3_attend.hip"
template <typename Load>
__device__ __forceinline__ void between(const float* a, float* out, Load&& load) {
  __shared__ __align__(16) float lds[3 * 64 * 4];
  using global_t = const __attribute__((address_space(1))) void;
  using local_t = __attribute__((address_space(3))) void;
  __builtin_amdgcn_global_load_lds((global_t*)(a + 4 * threadIdx.x), (local_t*)lds, 16, 0, 0);
  load();
  __builtin_amdgcn_global_load_lds((global_t*)(a + 4 * threadIdx.x + 256), (local_t*)lds, 16, 0, 0);
  q3::wait_loads<0>();
  __syncthreads();
  out[threadIdx.x] = lds[threadIdx.x];
}
extern "C" __global__ void probe_any(const float* a, float* out) {
  between(a, out, [&] { q3::load_lds(a + 4 * threadIdx.x, 1024u); });
}
extern "C" __global__ void probe_run(const float* a, float* out) {
  between(a, out, [&] { q3::load_lds(a, 16u * threadIdx.x, 1024u); });
}
"""


def test_the_compiler_knows_what_the_loads_write(tmp_path):
    from bit_fp8_codebook_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    (tmp_path / "probe.hip").write_text(PROBE)
    out = str(tmp_path / "probe.s")
    subprocess.run([hipcc, *build.COMMON, *build.DEVICE_FLAGS, "--cuda-device-only", "-S", str(tmp_path / "probe.hip"),
                    "-o", out], check=True, capture_output=True)
    text = open(out).read()
    for name in ("probe_any", "probe_run"):
        body = text[text.index(f"\n{name}:"):]
        lines = [x.strip() for x in body[:body.index("s_endpgm")].split("\n")]
        seen = [x for x in lines if re.match(r"s_\w+ m0,|global_load_lds", x)]
        loads = [i for i, x in enumerate(seen) if x.startswith("global_load_lds")]
        assert len(loads) == 3, seen
        assert all(i > 0 and " m0," in seen[i - 1] for i in loads), seen

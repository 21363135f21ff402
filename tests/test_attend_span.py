"""The positions that a tile of rows walks, from lengths and windows of every size,
on the host: the header that the attention kernels take them from, in a small
program of its own.  CPU only."""
import subprocess

import pytest

PROBE = r"""
#include <stdio.h>
#include "q3_span.h"
int main() {
  long long first, last, window, pages;
  int shift, step;
  while (scanf("%lld %lld %lld %lld %d %d", &first, &last, &window, &pages, &shift, &step) == 6) {
    const q3::Span s = q3::span_between((int)first, (int)last, (int)window, pages, shift);
    printf("%d %d %d %d\n", s.lo, s.hi, q3::first_of(s, step), q3::steps_of(s, step));
  }
}
"""
BIG = 2 ** 31 - 1
KEYS = 0x7FFFF000   # attention sees positions below it


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    from bit_fp8_codebook_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    d = tmp_path_factory.mktemp("span")
    (d / "probe.hip").write_text(PROBE)
    exe = str(d / "probe")
    subprocess.run([hipcc, *build.COMMON, *build.DEVICE_FLAGS, str(d / "probe.hip"), "-o", exe], check=True,
                   capture_output=True)

    def run(cases):
        text = "".join(" ".join(str(x) for x in c) + "\n" for c in cases)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout
        return [tuple(int(x) for x in line.split()) for line in out.splitlines()]
    return run


def _cases():
    lengths = [1, 2, 63, 64, 65, 127, 128, 129, 5000, 2 ** 30, KEYS - 65, KEYS - 1, KEYS, KEYS + 1, KEYS + 64, KEYS + 128,
               BIG - 4000, BIG - 128, BIG - 64, BIG - 1, BIG]
    tables = [(1, 0), (1, 4), (8, 4), (300, 6), (KEYS >> 10, 10), (1 << 21, 10), (1 << 31, 0), (1 << 40, 10)]
    for length in lengths:
        for new in (1, 2, 9, 130):
            for window in (0, 1, 2, 63, 64, 65, 127, 128, 4096, BIG):
                for pages, shift in tables:
                    for step in (64, 128):
                        yield length - new, length - 1, window, pages, shift, step


def test_every_walk_stays_in_32_bits_and_sees_what_it_should(walk):
    cases = list(_cases())
    answers = walk(cases)
    assert len(answers) == len(cases)
    for case, (lo, hi, begin, steps) in zip(cases, answers):
        first, last, window, pages, shift, step = case
        want_lo = max(0, first - window + 1) if window else 0
        want_hi = min(last + 1, pages << shift, KEYS)
        if want_lo >= want_hi:      # nothing is seen: nothing is walked
            assert hi == lo and steps == 0, case
        else:
            assert (lo, hi) == (want_lo, want_hi), case
            assert begin == lo - lo % step and begin + (steps - 1) * step < hi <= begin + steps * step, case
        assert 0 <= begin <= begin + steps * step <= BIG, case

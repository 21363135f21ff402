"""q3_logprobs and its backward pass at the ends of their arguments."""
import numpy as np
import pytest
import torch

from oracle import q3_attend as att
from paged_util import F32, cuda, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


def _coldest():
    """The smallest temperature whose log2(e) / t is finite in fp32, and the next below."""
    f32, log2e = np.float32, np.float32(1.4426950408889634)
    with np.errstate(over="ignore"):
        fine = lambda bits: np.isfinite(f32(1) / np.uint32(bits).view(f32) * log2e)  # noqa: E731
        lo, hi = 1, int(f32(1e-38).view(np.uint32))     # not fine, fine: positive floats order as their bits
        while hi - lo > 1:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if fine(mid) else (mid, hi)
    return float(np.uint32(hi).view(f32)), float(np.uint32(lo).view(f32))


@pytest.mark.parametrize("n", [7, 9001])
def test_the_coldest_temperature(q3, n):
    cold, below = _coldest()
    assert 4.2e-39 < cold < 4.3e-39
    rng = np.random.default_rng(31)
    m = 3
    l = (rng.integers(-8, 9, size=(m, n)) * 1e-39).astype(np.float32)     # differences of some temperatures
    l[2] = rng.normal(size=n).astype(np.float32)                          # and of all too many
    t = rng.integers(0, n, size=m).astype(np.int32)
    t[2] = int(l[2].argmax())
    for temperature in (cold, float(np.float32(cold * 1.5))):
        exact = 1 / float(np.float32(1) / np.float32(temperature))   # the kernel takes fp32's reciprocal
        r = q3.q3_logprobs(cuda(l), cuda(t), temperature)
        d = host(q3.q3_logprobs_backward(cuda(l), cuda(t), r.stats, torch.ones(m, device="cuda"), temperature=temperature,
                                         dtype=torch.float32))
        lp, h = host(r.logprobs), host(r.entropy)
        for i in range(m):
            want, ent, _, _ = att.logprobs(l[i], int(t[i]), exact)
            # 64 and the sum's roundings, and 8 of the log itself (a value of at most 4 + ln n)
            off = F32 * ((n + 8191) // 8192 * 16 + 72 + 8 * (4 + np.log(n)))
            assert abs(lp[i] - want) <= off, (i, lp[i], want)
            assert abs(h[i] - ent) <= 2 * off * (1 + np.log(n) + 4), (i, h[i], ent)
            # 1/T times [target] - p: p off by its log's error
            p = np.exp(att.log_softmax(l[i], exact))
            ref = ((np.arange(n) == t[i]) - p) / exact
            assert (np.abs(d[i] - ref) <= (2 * off * p + 4 * F32) / exact).all(), i
    for temperature in (below, 3e-39, 2.95e-39):
        with pytest.raises(q3.Q3Error):
            q3.q3_logprobs(cuda(l), cuda(t), temperature)
        with pytest.raises(q3.Q3Error):
            q3.q3_logprobs_backward(cuda(l), cuda(t), r.stats, torch.ones(m, device="cuda"), temperature=temperature)

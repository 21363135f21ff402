"""q3_logprobs and its backward pass against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import q3_attend as att
from paged_util import BF, F32, cuda, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


def _adds(n):
    """Roundings that a row's sums go through: 16 additions of 8192 logits in turn
    per thread, 9 + 4 + 10 levels of joins with a rescaling each, and the weight's
    own: two products, a difference, an exponential good to 2 (in all under 64)."""
    return (n + 8191) // 8192 * 16 + 64


def _off(n, logp):
    """How far a log probability may be: the sum's relative error, and the roundings
    of the difference and its scaling, relative to its size."""
    return F32 * (_adds(n) + 8 + 8 * np.abs(logp))


SHAPES = [(1, 1), (2, 2), (3, 7), (1, 63), (5, 100), (2, 1023), (1, 4096), (3, 8191), (2, 8192), (2, 8193), (1, 32000),
          (7, 50257), (2, 151936), (1100, 257), (1024, 9001)]


def _rows(rng, m, n, kind):
    l = rng.normal(size=(m, n)) * 3
    if kind == "ties":
        l = np.round(l)
        l[0] = 2.5          # all equal
        if m > 1:
            l[1] = np.where(np.arange(n) % 2, 0.0, -0.0)
    if kind == "masks":
        l[rng.random((m, n)) < 0.4] = -np.inf
        l[rng.random((m, n)) < 0.1] = np.nan
        l[0] = -np.inf      # nothing left
        if m > 1:
            l[1, rng.integers(0, n)] = np.inf
        if m > 2:
            l[2] = -3.4028234663852886e38   # the type's lowest is an ordinary logit
    if kind == "large":
        l = l * 1e4 + 3e5
    return l.astype(np.float32)


@pytest.mark.parametrize("kind", ["plain", "ties", "masks", "large"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rows(q3, shape, kind):
    m, n = shape
    rng = np.random.default_rng(m * 1000 + n)
    l = _rows(rng, m, n, kind)
    t = rng.integers(0, n, size=m).astype(np.int32)
    t[rng.random(m) < 0.2] = -1
    if m > 3:
        t[3] = n            # past the end: none
    top, temperature = int(rng.choice([0, 1, 3, 20, 32])), float(rng.choice([1.0, 0.7, 2.0]))
    r = q3.q3_logprobs(cuda(l), cuda(t), temperature, top)
    lp, h = host(r.logprobs), host(r.entropy)
    check = range(m) if m <= 16 else rng.choice(m, 16, replace=False)
    for i in check:
        # the kernel takes fp32's reciprocal of the temperature
        want = att.logprobs(l[i], int(t[i]), 1 / float(np.float32(1) / np.float32(temperature)), top)
        if np.isfinite(want[0]):
            assert abs(lp[i] - want[0]) <= _off(n, want[0]), i
        else:
            assert lp[i] == want[0], i
        # H = ln S - T / S: each weight times its log, with the same relative errors
        logp = att.log_softmax(l[i], temperature)
        live = logp[logp > -np.inf]
        spread = (np.exp(live) * (np.abs(live) + np.abs(live - live.max()))).sum() if len(live) else 0.0
        assert abs(h[i] - want[1]) <= F32 * (2 * _adds(n) + 16) * (1 + spread + np.log(n)), (i, h[i], want[1])
        if top:
            assert r.top_ids[i].tolist() == want[2].tolist(), i
            got, ref = host(r.top_logprobs[i]), want[3]
            fin = np.isfinite(ref)
            assert (got[~fin] == ref[~fin]).all() and (np.abs(got[fin] - ref[fin]) <= _off(n, ref[fin])).all(), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["plain", "ties", "masks", "large"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(q3, shape, kind, dtype):
    m, n = shape
    rng = np.random.default_rng(m * 1000 + n + 1)
    l = _rows(rng, m, n, kind)
    t = rng.integers(0, n, size=m).astype(np.int32)
    t[rng.random(m) < 0.2] = -1
    g, e = rng.normal(size=m).astype(np.float32), rng.normal(size=m).astype(np.float32)
    temperature = float(rng.choice([1.0, 0.5]))
    stats = q3.q3_logprobs(cuda(l), cuda(t), temperature).stats
    d = q3.q3_logprobs_backward(cuda(l), cuda(t), stats, cuda(g), cuda(e), temperature, dtype)
    assert d.dtype == dtype and d.shape == (m, n) and (m == 1 or d.stride(0) % 8 == 0)
    none = q3.q3_logprobs_backward(cuda(l), cuda(t), stats, None, None, temperature, dtype)
    assert not none.any()
    check = range(m) if m <= 16 else rng.choice(m, 16, replace=False)
    for i in check:
        ref = att.logprobs_backward(l[i], int(t[i]), float(g[i]), float(e[i]), temperature)
        got = host(d[i])
        logp = att.log_softmax(l[i], temperature)
        p, hh = np.exp(logp), att.entropy(logp)
        lp = np.where(logp > -np.inf, np.abs(logp), 0)
        # p is off by its log's error, the entropy by the bound of test_rows, (1 + H + ln n) large
        parts = p * (abs(g[i]) + abs(e[i]) * (lp + hh + 1)) + (np.arange(n) == t[i]) * abs(g[i])
        off = (F32 * (2 * _adds(n) + 32 + 8 * lp) * (2 + np.log(n))) * parts / temperature
        bound = off + (BF if dtype == torch.bfloat16 else F32) * np.abs(ref) + 1e-37
        bad = ~(np.abs(got - ref) <= bound * 1.01)
        assert not bad.any(), (i, np.argwhere(bad)[:3].ravel(), got[bad][:3], ref[bad][:3])


def test_backward_against_differences(q3):
    rng = np.random.default_rng(9)
    l, t = (rng.normal(size=(2, 12)) * 2).astype(np.float32), np.array([3, -1], np.int32)
    g, e = np.array([0.7, 0.4], np.float32), np.array([-0.3, 1.1], np.float32)
    d = q3.q3_logprobs_backward(cuda(l), cuda(t), q3.q3_logprobs(cuda(l), cuda(t)).stats, cuda(g), cuda(e),
                                dtype=torch.float32)
    for i in np.ndindex(l.shape):
        def f(step):
            row = l[i[0]].astype(np.float64)
            row[i[1]] += step
            r = att.logprobs(row, int(t[i[0]]))
            return float(g[i[0]]) * r[0] + float(e[i[0]]) * r[1]
        # the quotient is good to 1e-8, the gradient to a few roundings of values below 4
        assert abs(float(d[i]) - (f(1e-5) - f(-1e-5)) / 2e-5) < 1e-5, i


def test_pitched_rows_and_in_place(q3):
    rng = np.random.default_rng(10)
    m, n = 5, 1003
    l, t = cuda((rng.normal(size=(m, n)) * 3).astype(np.float32)), cuda(rng.integers(0, n, size=m).astype(np.int32))
    g, e = cuda(rng.normal(size=m).astype(np.float32)), cuda(rng.normal(size=m).astype(np.float32))
    wide = torch.full((m, n + 6), float("nan"), device="cuda")
    wide[:, 1:n + 1] = l
    odd = wide[:, 1:n + 1]                                  # rows that start 4 bytes off
    a, b = q3.q3_logprobs(l, t, 0.9, 7), q3.q3_logprobs(odd, t, 0.9, 7)
    for x, y in ((a.logprobs, b.logprobs), (a.entropy, b.entropy), (a.stats, b.stats), (a.top_ids, b.top_ids),
                 (a.top_logprobs, b.top_logprobs)):
        assert torch.equal(x, y)
    for dtype in (torch.float32, torch.bfloat16):
        want = q3.q3_logprobs_backward(l, t, a.stats, g, e, 0.9, dtype)
        out = torch.full((m, n + 3), 9.0, dtype=dtype, device="cuda")
        q3.q3_logprobs_backward(odd, t, a.stats, g, e, 0.9, dlogits=out[:, 1:n + 1])
        assert torch.equal(out[:, 1:n + 1], want) and (out[:, 0] == 9).all() and (out[:, n + 1:] == 9).all()
    want = q3.q3_logprobs_backward(l, t, a.stats, g, e, 0.9, torch.float32)
    same = l.clone()
    assert q3.q3_logprobs_backward(same, t, a.stats, g, e, 0.9, dlogits=same) is same and torch.equal(same, want)


def test_clumped_candidates(q3):
    # rising rows (every chunk beats the list), one lane's columns holding all the best, many equal at the border
    n = 40000
    rise = np.arange(n, dtype=np.float32)
    lane = np.zeros(n, np.float32)
    lane[:4] = 9
    lane[2048:2052] = 8     # the same thread's next four
    lane[4096:4100] = 7
    border = np.full(n, 1.0, np.float32)
    border[::7] = 2.0
    border[5] = 3.0
    fall = -rise
    l = np.stack([rise, lane, border, fall])
    r = q3.q3_logprobs(cuda(l), cuda(np.zeros(4, np.int32)), 1.0, 32)
    for i in range(4):
        assert r.top_ids[i].tolist() == att.logprobs(l[i], 0, 1.0, 32)[2].tolist(), i


def test_more_rows_than_one_launch(q3):
    m, n = 65535 * 2 + 3, 33
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(m, n, generator=g, device="cuda")
    t = (torch.arange(m, device="cuda") % n).int()
    d = torch.ones(m, device="cuda")
    r = q3.q3_logprobs(l, t, 1.0, 2)
    at = [0, 65534, 65535, 131070, m - 1]
    s = q3.q3_logprobs(l[at].contiguous(), t[at].contiguous(), 1.0, 2)
    for a, b in ((r.logprobs, s.logprobs), (r.entropy, s.entropy), (r.top_ids, s.top_ids), (r.stats, s.stats)):
        # few rows are one block each too: the same sums
        assert torch.equal(a[at], b)
    whole = q3.q3_logprobs_backward(l, t, r.stats, d, d)
    few = q3.q3_logprobs_backward(l[at].contiguous(), t[at].contiguous(), s.stats, d[at].contiguous(), d[at].contiguous())
    assert torch.equal(whole[at], few)
    lp = torch.log_softmax(l.double(), 1).gather(1, t.long().view(m, 1)).view(m)
    assert (lp - r.logprobs.double()).abs().max() < 1e-5   # 80 + 8 * 12 roundings of 2^-24


def test_equal_calls_give_equal_bits(q3):
    rng = np.random.default_rng(11)
    l, t = cuda((rng.normal(size=(3, 70001)) * 2).astype(np.float32)), cuda(np.array([5, 6, 7], np.int32))
    a, b = q3.q3_logprobs(l, t, 1.0, 20), q3.q3_logprobs(l, t, 1.0, 20)
    for x, y in ((a.logprobs, b.logprobs), (a.stats, b.stats), (a.top_ids, b.top_ids), (a.top_logprobs, b.top_logprobs)):
        assert torch.equal(x, y)

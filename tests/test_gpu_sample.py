"""Sampling on the GPU against the fp64 oracle: tokens are equal, logprobs agree
to fp32.  Kernel weights are integers of 2^-44, the oracle's are fp64; they
pick different tokens only where u lies within n * 2^-45 of a running sum's
border, which the seeded rows here do not."""
import numpy as np
import pytest
import torch

from oracle import q3_block as blk

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def check(q3, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, **kw):
    dev = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a), dtype=t).cuda()  # noqa: E731
    lg = logits if isinstance(logits, torch.Tensor) else torch.as_tensor(np.asarray(logits), dtype=torch.float32)
    lg = lg.cuda() if not lg.is_cuda else lg
    f = torch.float32
    host = [None if a is None else np.asarray(dev(a, t).cpu().double())
            for a, t in ((u, f), (temperature, f), (top_k, torch.int32), (top_p, f), (min_p, f))]
    tok, lp = q3.q3_sample(lg, dev(u, f), dev(temperature, f), dev(top_k, torch.int32), dev(top_p, f), dev(min_p, f),
                           **kw)
    tok, lp, rows = tok.cpu().numpy(), lp.cpu().numpy(), lg.cpu().double().numpy()
    for i in range(len(rows)):
        at = lambda a, d: d if a is None else a[i]  # noqa: E731
        t, p = blk.sample(rows[i], host[0][i], at(host[1], 1.0), int(at(host[2], 0)), at(host[3], 1.0),
                          at(host[4], 0.0))
        assert tok[i] == t, (i, tok[i], t)
        # fp32 rounding of the result and 2^-45 for each of n weights against a sum of at least 1
        assert lp[i] == p or abs(lp[i] - p) <= 2.0 ** -23 * abs(p) + 2e-7, (i, lp[i], p)
    return tok


def rows(m, n, spread=2.0, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.normal(size=(m, n)) * spread).astype(np.float32), rng.random(m).astype(np.float32)


@pytest.mark.parametrize("n", [1, 2, 7, 63, 64, 1000, 1023, 1024, 1025, 4097, 32000, 50257, 151936])
def test_sizes(q3, n):
    l, u = rows(5, n, seed=n)
    check(q3, l, u)
    check(q3, l, u, top_p=[0.1, 0.5, 0.9, 0.99, 0.0])
    check(q3, l, u, top_k=[1, 2, 5, n, n + 7])
    check(q3, l, u, min_p=[0.5, 0.1, 0.01, 1e-6, 1.0])
    check(q3, l, u, [0.3, 1.0, 2.0, 0.0, 0.7], [40, 0, 3, 9, 1000], [0.9, 0.8, 1.0, 0.2, 0.95], [0, 0.05, 0.02, 0, 0.1])


@pytest.mark.parametrize("m", [1, 2, 17, 64, 300, 700])
def test_batches(q3, m):
    n = 3000
    l, u = rows(m, n, seed=m)
    rng = np.random.default_rng(m)
    check(q3, l, u, 0.2 + rng.random(m), rng.integers(0, 60, m), 0.3 + 0.8 * rng.random(m), 0.1 * rng.random(m) - 0.02)


@pytest.mark.parametrize("spread", [0.0, 1e-6, 1e-3, 0.05, 10.0, 1000.0])
def test_spreads(q3, spread):
    # from all equal (everything at the border) to one entry with weight
    l, u = rows(6, 9000, spread, seed=11)
    check(q3, l, u)
    check(q3, l, u, top_p=[0.01, 0.3, 0.5, 0.9, 0.999, 0.9999999])
    check(q3, l, u, top_k=[1, 7, 100, 3000, 8999, 9000])
    check(q3, l, u, None, [5000] * 6, [0.5] * 6, [0.9, 0.999, 1.0, 0.1, 1e-3, 0.0])


def test_ties(q3):
    rng = np.random.default_rng(5)
    l = np.round(rng.normal(size=(8, 20000)) * 2).astype(np.float32)   # a few values, thousands of entries each
    u = rng.random(8).astype(np.float32)
    check(q3, l, u, top_k=[1, 10, 100, 1000, 5000, 9999, 15000, 19999])
    check(q3, l, u, top_p=[0.001, 0.1, 0.3, 0.5, 0.7, 0.9, 0.99, 0.9999])
    check(q3, l, u, 0.5 + rng.random(8), rng.integers(1, 20000, 8), rng.random(8), 0.3 * rng.random(8))


def longer(l, n):
    """The same rows with masked entries behind them, up to n."""
    return np.concatenate([l, np.full((len(l), n - l.shape[1]), -INF, np.float32)], 1)


@pytest.mark.parametrize("n", [20480, 20481, 65536, 65537, 131072])
def test_rows_in_one_block_and_in_several(q3, n):
    # spreads, ties and masks at both sides of the length where a row is split over blocks
    rng = np.random.default_rng(n)
    l, u = rows(8, 9000, seed=n)
    l[1] = np.round(l[1])
    l[2] = 1.5
    l[3, rng.random(9000) < 0.9] = -INF
    l[4, rng.random(9000) < 0.5] = np.nan
    l[5, [7, 400, 8999]] = INF
    l[6] = -INF
    l[7] *= 100
    long = np.concatenate([longer(l, n), rows(4, n, seed=1)[0]])
    u = rng.random(12).astype(np.float32)
    u[3], u[9] = 1.0, 0.0
    check(q3, long, u)
    check(q3, long, u, top_k=[1, 50, 3000, 9, 1000, 2, 3, 1, 40, n - 1, n // 2, 5])
    check(q3, long, u, top_p=rng.random(12))
    check(q3, long, u, 0.3 + rng.random(12), rng.integers(0, 4000, 12), 0.2 + rng.random(12), 0.1 * rng.random(12))
    tok = check(q3, long, u, temperature=np.zeros(12))
    assert tok[6] == -1


def test_many_long_rows(q3):
    for n in (30000, 65536, 65537):
        l, u = rows(256, n, seed=n)
        check(q3, l, u, top_k=[0, 30] * 128, top_p=[0.9, 1.0, 0.5, 0.99] * 64)


def test_equal_weights_draw_evenly(q3):
    # dyadic sums are exact on both sides: u = i/n picks entry i
    n = 4096
    u = np.arange(0, n, 37, dtype=np.float32) / n
    tok = check(q3, np.zeros((len(u), n), np.float32), u)
    assert (tok == np.arange(0, n, 37)).all()


def test_masks(q3):
    l, u = rows(9, 5000, seed=2)
    rng = np.random.default_rng(9)
    l[0] = -INF
    l[1] = np.nan
    l[2, :] = -INF
    l[2, 4321] = -3.5
    l[3, rng.random(5000) < 0.9] = -INF
    l[4, rng.random(5000) < 0.5] = np.nan
    l[5, [7, 400, 4999]] = INF
    l[6, :] = -3.4028235e38
    l[6, [5, 6]] = 1.0
    l[7, :] = -3.4028235e38          # the type's lowest value everywhere: all equal
    l[8, ::2] = 3.0e38
    l[8, 1::2] = -3.0e38
    for kw in (dict(), dict(top_k=[3] * 9), dict(top_p=[0.6] * 9), dict(min_p=[0.05] * 9),
               dict(temperature=[0.0] * 9), dict(top_k=[50] * 9, top_p=[0.9] * 9, min_p=[0.01] * 9)):
        tok = check(q3, l, u, **kw)
        assert tok[0] == -1 and tok[1] == -1 and tok[2] == 4321 and tok[5] in (7, 400, 4999)


def test_settings_at_their_ends(q3):
    l, u = rows(8, 2000, seed=3)
    nan = float("nan")
    check(q3, l, [0.0, 1.0, 2.0, -1.0, nan, 0.99999994, 1e-30, 0.5])
    check(q3, l, u, temperature=[nan, INF, 1e30, 1e-30, 1e-45, -1.0, 0.0, 1e-3])
    check(q3, l, u, top_p=[nan, INF, -1.0, 0.0, 1.0, 1e-30, 0.99999994, 2.0])
    check(q3, l, u, min_p=[nan, INF, -1.0, 0.0, 1.0, 1e-30, 0.99999994, 2.0])
    check(q3, l, u, top_k=[-5, 0, 1, 2000, 1999, 2001, 2147483647, -2147483648])


def test_offset_logits(q3):
    # far from zero the steps between logits are coarse: many equal entries
    l, u = rows(6, 8000, seed=4)
    for off in (1e3, -1e5, 1e7):
        check(q3, l + np.float32(off), u, None, [50, 500, 5000, 0, 0, 7], [0.9, 1.0, 0.5, 0.5, 0.99, 1.0],
              [0.0, 0.1, 0.0, 0.2, 0.001, 0.05])


def test_pitched_rows_outputs_and_workspace(q3):
    l, u = rows(4, 3000, seed=6)
    wide = torch.full((4, 3100), INF, device="cuda")     # what stands behind the rows is not read
    wide[:, :3000] = torch.from_numpy(l).cuda()
    ws = q3.sample_workspace(4, 3000, "cuda")
    ws.fill_(255)
    tok, lp = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    a = check(q3, wide[:, :3000], u, top_p=[0.9] * 4, workspace=ws, tokens=tok, logprobs=lp)
    b = check(q3, l, u, top_p=[0.9] * 4, workspace=ws)
    assert (a == b).all() and (tok.cpu().numpy() == a).all()
    with pytest.raises(q3.Q3Error):
        q3.q3_sample(wide[:, :3000], tok.float(), workspace=ws[:ws.numel() // 2])
    with pytest.raises(q3.Q3Error):
        q3.q3_sample(torch.zeros(1, (1 << 19) + 1, device="cuda"), torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        q3.q3_sample(wide, torch.zeros(4), top_k=torch.zeros(4, device="cuda"))


def test_largest_vocabulary(q3):
    l, u = rows(2, 1 << 19, seed=8)
    check(q3, l, u, top_p=[0.9, 0.999])
    check(q3, np.zeros((2, 1 << 19), np.float32), u, top_p=[0.25, 1.0])


@pytest.mark.parametrize("n", [4000, 40000])
def test_captured_and_replayed(q3, n):
    # new logits, numbers and settings under the same graph; other work in between
    l = torch.randn(5, n, device="cuda")
    u = torch.rand(5, device="cuda")
    p = torch.full((5,), 0.9, device="cuda")
    ws = q3.sample_workspace(5, n, "cuda")
    tok, lp = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, device="cuda")
    q3.q3_sample(l, u, top_p=p, workspace=ws, tokens=tok, logprobs=lp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q3.q3_sample(l, u, top_p=p, workspace=ws, tokens=tok, logprobs=lp)
    for i in range(4):
        l.copy_(torch.randn(5, n, device="cuda") * (i + 0.5))
        u.copy_(torch.rand(5, device="cuda"))
        p.fill_(0.5 + 0.15 * i)
        g.replay()
        torch.cuda.synchronize()
        a, b = tok.clone(), lp.clone()
        t2, l2 = q3.q3_sample(l, u, top_p=p)
        assert torch.equal(a, t2) and torch.equal(b, l2)
        torch.zeros(1000, device="cuda").sum().item()


def test_another_stream(q3):
    l, u = rows(3, 20000, seed=12)
    lg, uu = torch.from_numpy(l).cuda(), torch.from_numpy(u).cuda()
    want, _ = q3.q3_sample(lg, uu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, _ = q3.q3_sample(lg, uu)
    s.synchronize()
    assert torch.equal(want, got)

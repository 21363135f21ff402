"""q3_qk_norm_rope and its backward pass against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import q3_attend as att
from paged_util import BF, F32, Paged, cuda, host

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


def _heads(x, hq, hk, d):
    x = x.reshape(len(x), hq + 2 * hk, d)
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def _check(got, ref, near, what):
    """bf16 results: half a step, and what the fp32 evaluation can be off: the norm's
    sum and root 24 roundings, the angle, its sine and the two products 8, of the
    pair's size `near`.  (A sum of d <= 256 squares in a tree of depth 8 after 8 in
    turn, a division, an addition, a root good to 2, two products: under 24.)"""
    got = host(got).reshape(ref.shape)
    bound = BF * np.abs(ref) + 32 * F32 * near + 1e-38
    bad = np.abs(got - ref) > bound * (1 + BF)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def _near(x, w):
    """A bound of both values of a pair: the head's largest value after its norm."""
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * w
    return 2 * np.abs(n).max(-1, keepdims=True)


CASES = [  # m, hq, hk, d, rotated, interleaved, norms of (q, k)
    (1, 1, 1, 16, 16, False, (True, True)), (3, 4, 2, 64, 64, False, (True, True)),
    (5, 32, 8, 128, 128, False, (True, True)), (7, 3, 1, 80, 80, True, (True, False)),
    (17, 6, 3, 96, 40, False, (False, True)), (9, 5, 5, 112, 56, True, (True, True)),
    (4, 2, 1, 256, 256, False, (True, True)), (6, 16, 2, 192, 6, False, (True, True)),
    (2, 7, 2, 32, 0, False, (True, True)), (1500, 2, 1, 48, 48, True, (False, False)), (11, 40, 3, 176, 2, True, (True, True)),
    (1025, 3, 2, 64, 34, False, (True, True)),
]


def _inputs(case, seed=0):
    m, hq, hk, d, turned, _, norms = case
    rng = np.random.default_rng(seed)
    qkv = rng.normal(size=(m, (hq + 2 * hk) * d)).astype(np.float32)
    qkv[rng.integers(0, m)] *= 1e-4   # where eps counts
    freq = (10000.0 ** (-np.arange(turned // 2) * 2 / max(turned, 1))).astype(np.float32)
    w = [(1 + 0.3 * rng.normal(size=d)).astype(np.float32) if n else None for n in norms]
    pos = rng.integers(0, 300000, size=m).astype(np.int32)
    pos[0] = 2 ** 31 - 1   # the farthest
    return rng, qkv, freq, w, pos


@pytest.mark.parametrize("case", CASES)
def test_rows(q3, case):
    m, hq, hk, d, turned, pairs, _ = case
    _, qkv, freq, w, pos = _inputs(case)
    dw = [None if x is None else cuda(x) for x in w]
    got = q3.q3_qk_norm_rope(cuda(qkv), hq, hk, cuda(freq) if turned else None, cuda(pos), *dw, eps=EPS,
                             interleaved=pairs)
    x = _heads(qkv.astype(np.float64), hq, hk, d)
    for g, h, ww, name in ((got[0], x[0], w[0], "q"), (got[1], x[1], w[1], "k")):
        ww = None if ww is None else ww.astype(np.float64)
        ref = att.head_norm_rope(h, ww, pos.astype(np.float64), freq.astype(np.float64), EPS, pairs)
        _check(g, ref, _near(h, ww), name)
    assert torch.equal(got[2], cuda(qkv)[:, (hq + hk) * d:].to(torch.bfloat16))


@pytest.mark.parametrize("case", CASES[:8])
def test_equal_calls_give_equal_bits_with_pitched_rows(q3, case):
    m, hq, hk, d, turned, pairs, _ = case
    rng, qkv, freq, w, pos = _inputs(case, 1)
    dw = [None if x is None else cuda(x) for x in w]
    n = qkv.shape[1]
    wide = torch.full((m, n + 12), float("nan"), device="cuda")
    wide[:, :n] = cuda(qkv)
    out = [torch.full((m, h * d + 8), -5.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hk, hk)]
    args = (hq, hk, cuda(freq) if turned else None, cuda(pos), *dw)
    a = q3.q3_qk_norm_rope(cuda(qkv), *args, interleaved=pairs)
    q3.q3_qk_norm_rope(wide[:, :n], *args, interleaved=pairs, q=out[0][:, :-8], k=out[1][:, :-8], v=out[2][:, :-8])
    for x, y in zip(a, out):
        assert torch.equal(x, y[:, :-8]) and (y[:, -8:] == -5).all()


@pytest.mark.parametrize("page", [1, 4, 16, 1024])
@pytest.mark.parametrize("shape", [(4, 2, 64), (3, 1, 128), (8, 4, 80)])
def test_into_a_cache(q3, page, shape):
    hq, hk, d = shape
    rng = np.random.default_rng(2)
    # a decoding token, a prompt, no new token, drafted ones; positions before 0; a table too short
    p = Paged(rng, [1, 37, 0, 8, 5, 3], [50, 37, 12, 100, 2, 0], hk, d, page, gap=16)
    cache, batch = p.on_device(q3)
    m = p.m + 2   # two rows of no sequence
    qkv = rng.normal(size=(m, (hq + 2 * hk) * d)).astype(np.float32)
    freq = (1e6 ** (-np.arange(d // 2) * 2 / d)).astype(np.float32)
    w = [(1 + 0.3 * rng.normal(size=d)).astype(np.float32) for _ in range(2)]
    q = torch.full((m, hq * d), 7.0, dtype=torch.bfloat16, device="cuda")
    before = cache.k.clone(), cache.v.clone()
    got, k, v = q3.q3_qk_norm_rope(cuda(qkv), hq, hk, cuda(freq), None, cuda(w[0]), cuda(w[1]), cache=cache,
                                   batch=batch, q=q)
    assert got is q and k is None and v is None and (q[p.m:] == 7).all()
    where = att.places(p.start, p.length, m)
    x = _heads(qkv.astype(np.float64), hq, hk, d)
    pos = where[:p.m, 1].astype(np.float64)
    wd = [a.astype(np.float64) for a in w]
    refs = [att.head_norm_rope(x[i][:p.m], wd[i], pos, freq.astype(np.float64), EPS) for i in (0, 1)]
    _check(q[:p.m], refs[0], _near(x[0][:p.m], wd[0]), "q")
    written = torch.zeros(cache.k.shape[0], p.page, dtype=torch.bool)
    for i in range(p.m):
        f = att.find(p.table, cache.k.shape[0], page, *where[i])
        if f is None:
            continue
        written[f] = True
        _check(cache.k[f[0], :, f[1]], refs[1][i], _near(x[1][i], wd[1]), ("k", i))
        assert torch.equal(cache.v[f[0], :, f[1]], cuda(qkv[i]).view(-1, d)[hq + hk:].to(torch.bfloat16))
    assert written.sum() == 1 + 37 + 8 + 2
    keep = ~written.cuda()
    for now, old in ((cache.k, before[0]), (cache.v, before[1])):
        assert torch.equal(now.transpose(1, 2)[keep], old.transpose(1, 2)[keep])
    # given positions turn the rows; their places stay the batch's
    other = cuda(np.arange(m).astype(np.int32) + 1000)
    q3.q3_qk_norm_rope(cuda(qkv), hq, hk, cuda(freq), other, cuda(w[0]), cuda(w[1]), cache=cache, batch=batch, q=q)
    rows = q3.q3_qk_norm_rope(cuda(qkv), hq, hk, cuda(freq), other, cuda(w[0]), cuda(w[1]))
    assert torch.equal(q[:p.m], rows[0][:p.m])
    f = att.find(p.table, cache.k.shape[0], page, *where[0])
    assert torch.equal(cache.k[f[0], :, f[1]].reshape(-1), rows[1][0])


def test_broken_tables_write_nothing(q3):
    rng = np.random.default_rng(3)
    p = Paged(rng, [4, 4], [20, 20], 2, 64, 16)
    cache, batch = p.on_device(q3)
    qkv = cuda(rng.normal(size=(8, 8 * 64)).astype(np.float32))
    before = cache.k.clone(), cache.v.clone()
    pages = cache.k.shape[0]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    big = 2 ** 31 - 1
    for start, length, entry in ((i32(0, 4, 8), i32(20, 20), pages), (i32(0, 4, 8), i32(20, 20), -1),
                                 (i32(0, 4, 8), i32(20, 20), big), (i32(0, 4, 8), i32(20, 20), -big),
                                 (i32(0, 4, 8), i32(big, 300), 0), (i32(0, 4, 8), i32(-5, -big), 0),
                                 (i32(8, 8, 8), i32(20, 20), 0), (i32(big, 5, -big), i32(20, 20), pages)):
        table = torch.full((2, 2), entry, dtype=torch.int32, device="cuda")
        q3.q3_qk_norm_rope(qkv, 4, 2, None, cache=cache, batch=q3.PagedBatch(start, length, table))
    torch.cuda.synchronize()
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])


@pytest.mark.parametrize("b", [1, 63, 64, 65, 4095, 4200])
def test_many_sequences(q3, b):
    # one token each but for every fifth sequence; the search asks 64 entries a step
    new = [0 if s % 5 == 4 else 1 for s in range(b)]
    length = [(3 * s) % 7 + n for s, n in zip(range(b), new)]
    rng = np.random.default_rng(4)
    p = Paged(rng, new, length, 1, 16, 8)
    cache, batch = p.on_device(q3)
    qkv = rng.normal(size=(p.m, 3 * 16)).astype(np.float32)
    q3.q3_qk_norm_rope(cuda(qkv), 1, 1, None, cache=cache, batch=batch)
    v = cache.v.cpu()
    bits = torch.from_numpy(qkv)[:, 32:].to(torch.bfloat16)
    for i, (s, pos) in enumerate(att.places(p.start, p.length, p.m)):
        assert torch.equal(v[p.table[s, pos // 8], 0, pos % 8], bits[i]), (i, s)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", CASES)
def test_backward(q3, case, dtype):
    m, hq, hk, d, turned, pairs, _ = case
    rng, qkv, freq, w, pos = _inputs(case, 5)
    grads = [cuda(rng.normal(size=(m, h * d)).astype(np.float32)).to(dtype) for h in (hq, hk, hk)]
    g = q3.q3_qk_norm_rope_backward(cuda(qkv), hq, hk, cuda(freq) if turned else None, cuda(pos), *grads,
                                    *[None if x is None else cuda(x) for x in w], eps=EPS, interleaved=pairs)
    x = _heads(qkv.astype(np.float64), hq, hk, d)
    out = _heads(host(g.dqkv), hq, hk, d)
    for i, dw in ((0, g.dq_weight), (1, g.dk_weight)):
        ww = None if w[i] is None else w[i].astype(np.float64)
        gi = host(grads[i]).reshape(m, -1, d)
        dx, dweight = att.head_norm_rope_backward(x[i], gi, ww, pos.astype(np.float64), freq.astype(np.float64), EPS, pairs)
        # the parts of dx before they cancel: s |a| and s |h| mean |a h|
        size = 2 * np.abs(gi).max(-1, keepdims=True)
        if ww is not None:
            s = 1 / np.sqrt((x[i] ** 2).mean(-1, keepdims=True) + EPS)
            a, h = size * np.abs(ww), np.abs(x[i] * s)
            size = s * (a + h * (a * h).mean(-1, keepdims=True))
            # a sum over tokens and heads: up to m hq / 32 + 96 additions in turn of terms good to 32
            scale = (2 * np.abs(gi).max(-1, keepdims=True) * h).sum((0, 1))
            off = np.abs(host(dw) - dweight)
            assert (off <= (128 + m * x[i].shape[1] / 32) * F32 * scale).all(), ("dw", i, off.max())
        else:
            assert dw is None
        bound = BF * np.abs(dx) + 64 * F32 * size + 1e-38
        bad = np.abs(out[i] - dx) > bound * (1 + BF)
        assert not bad.any(), (i, np.argwhere(bad)[:4], out[i][bad][:4], dx[bad][:4])
    assert torch.equal(g.dqkv[:, (hq + hk) * d:], grads[2].to(torch.bfloat16))
    again = q3.q3_qk_norm_rope_backward(cuda(qkv), hq, hk, cuda(freq) if turned else None, cuda(pos), *grads,
                                        *[None if x is None else cuda(x) for x in w], eps=EPS, interleaved=pairs)
    for a, b in ((g.dqkv, again.dqkv), (g.dq_weight, again.dq_weight), (g.dk_weight, again.dk_weight)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_backward_against_differences(q3):
    # the forward in fp64 by the oracle, stepped; the kernel's gradient beside it
    m, hq, hk, d = 2, 2, 1, 16
    rng = np.random.default_rng(6)
    qkv = rng.normal(size=(m, 4 * d)).astype(np.float32)
    w = (1 + 0.3 * rng.normal(size=d)).astype(np.float32)
    freq, pos = np.array([1.0, 0.1, 0.01], np.float32), np.array([5, 70001], np.int32)
    g = [rng.normal(size=(m, h * d)).astype(np.float32) for h in (hq, hk, hk)]
    got = q3.q3_qk_norm_rope_backward(cuda(qkv), hq, hk, cuda(freq), cuda(pos), *[cuda(x) for x in g], cuda(w), cuda(w))

    def f(x):
        a = _heads(x, hq, hk, d)
        o = [att.head_norm_rope(a[i], w.astype(np.float64), pos.astype(np.float64), freq.astype(np.float64), EPS)
             for i in (0, 1)] + [a[2]]
        return sum((y.reshape(m, -1) * z).sum() for y, z in zip(o, g))
    base = qkv.astype(np.float64)
    for i in np.ndindex(base.shape):
        up, dn = base.copy(), base.copy()
        up[i] += 1e-5
        dn[i] -= 1e-5
        num = (f(up) - f(dn)) / 2e-5
        # the quotient is good to 1e-7; dqkv is rounded to bf16
        assert abs(float(got.dqkv[i]) - num) <= BF * abs(num) * 1.01 + 2e-5, i


def test_missing_gradients_are_zero(q3):
    rng = np.random.default_rng(7)
    m, hq, hk, d = 3, 4, 2, 64
    qkv, freq = cuda(rng.normal(size=(m, 8 * d)).astype(np.float32)), cuda(np.ones(32, np.float32))
    pos, w = cuda(np.arange(m, dtype=np.int32)), cuda(np.ones(d, np.float32))
    full = [cuda(rng.normal(size=(m, h * d)).astype(np.float32)) for h in (hq, hk, hk)]
    for skip in range(3):
        some = [None if i == skip else t for i, t in enumerate(full)]
        zero = [torch.zeros_like(t) if i == skip else t for i, t in enumerate(full)]
        a = q3.q3_qk_norm_rope_backward(qkv, hq, hk, freq, pos, *some, w, w)
        b = q3.q3_qk_norm_rope_backward(qkv, hq, hk, freq, pos, *zero, w, w)
        assert torch.equal(a.dqkv, b.dqkv) and torch.equal(a.dq_weight, b.dq_weight) and torch.equal(a.dk_weight, b.dk_weight)
    none = q3.q3_qk_norm_rope_backward(qkv, hq, hk, freq, pos)
    assert (none.dqkv == 0).all() and none.dq_weight is None


def test_one_tokens_values_stay_its_own(q3):
    rng = np.random.default_rng(8)
    m, hq, hk, d = 6, 4, 2, 80
    qkv = rng.normal(size=(m, 8 * d)).astype(np.float32)
    freq, pos = cuda(np.ones(40, np.float32)), cuda(np.arange(m, dtype=np.int32))
    w = cuda(np.ones(d, np.float32))
    clean = q3.q3_qk_norm_rope(cuda(qkv), hq, hk, freq, pos, w, w)
    dirty = qkv.copy()
    dirty[2, 3 * d + 5], dirty[4, 4 * d] = np.nan, np.inf   # head 3 of token 2, key head 0 of token 4
    got = q3.q3_qk_norm_rope(cuda(dirty), hq, hk, freq, pos, w, w)
    for a, b, hit in ((clean[0], got[0], (2, 3)), (clean[1], got[1], (4, 0))):
        same = torch.ones(m, a.shape[1] // d, dtype=torch.bool)
        same[hit] = False
        same = same.cuda()
        assert torch.equal(a.view(m, -1, d)[same], b.view(m, -1, d)[same])


def test_more_rows_than_one_launch(q3):
    # 2^22 rows go in one launch; the last ones are of the second
    m, d = (1 << 22) + 3, 16
    qkv = torch.zeros(m, 3 * d, device="cuda")
    tail = torch.arange(5 * 48, device="cuda", dtype=torch.float32).view(5, 48) / 16
    qkv[-5:] = tail
    pos = torch.zeros(m, dtype=torch.int32, device="cuda")
    pos[-5:] = 3
    freq = torch.ones(8, device="cuda")
    q, k, v = q3.q3_qk_norm_rope(qkv, 1, 1, freq, pos)
    small = q3.q3_qk_norm_rope(tail, 1, 1, freq, pos[-5:].clone())
    assert torch.equal(q[-5:], small[0]) and torch.equal(k[-5:], small[1]) and torch.equal(v[-5:], small[2])
    assert not q[:-5].any()

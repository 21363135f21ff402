"""Pins of the oracle of the operators between and behind the products: its
gradients against central differences of its forward formulas, its sampler
against hand-worked rows and a brute-force reading of the rules."""
import itertools
import math

import numpy as np
import pytest

from oracle import q3_block as blk


def _diff(f, x, i, d):
    up, dn = x.copy(), x.copy()
    up[i] += d
    dn[i] -= d
    return (f(up) - f(dn)) / (2 * d)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_slope_is_the_difference_quotient(act):
    z = np.linspace(-9, 9, 181)
    d = 1e-5
    num = (blk.act(act, z + d) - blk.act(act, z - d)) / (2 * d)
    # error of a central difference: d^2/6 |f'''| + 2^-53 |f| / d < 1e-9 here
    assert np.abs(num - blk.act_slope(act, z)).max() < 1e-9


def test_activation_values():
    assert blk.act("silu", 0.0) == 0 and abs(blk.act("silu", 1.0) - 1 / (1 + math.exp(-1))) < 1e-15
    assert abs(blk.act("gelu", 1.0) - 0.8411919906082768) < 1e-12
    for z in (-3.0, -0.5, 0.5, 3.0):   # the tanh form as it is written
        t = math.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        assert abs(blk.act("gelu", z) - 0.5 * z * (1 + t)) < 1e-14
    # far out on the left 1 + tanh would be 0; the value is z e^v
    v = 2 * math.sqrt(2 / math.pi) * (-8 - 0.044715 * 512)
    assert abs(blk.act("gelu", -8.0) / (-8 * math.exp(v)) - 1) < 1e-12


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gradient(act):
    rng = np.random.default_rng(0)
    w, x, dh = rng.normal(size=(12, 7)) * 0.5, rng.normal(size=(3, 7)), rng.normal(size=(3, 6))
    _, pre = blk.glu(w, x, act)
    dx = blk.glu_backward(pre, dh, act) @ w
    f = lambda v: (blk.glu(w, v, act)[0] * dh).sum()  # noqa: E731
    for i in itertools.product(range(3), range(7)):
        assert abs(_diff(f, x, i, 1e-5) - dx[i]) < 1e-8


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "row", "full"])
def test_norm_gradient(post, gate):
    rng = np.random.default_rng(1)
    m, n = 3, 5
    v = {"r": rng.normal(size=(m, n)), "pre_w": rng.normal(size=n), "y": rng.normal(size=(m, n)),
         "post_w": rng.normal(size=n) if post else None,
         "gate": {None: None, "row": rng.normal(size=n), "full": rng.normal(size=(m, n))}[gate]}
    dx, dr = rng.normal(size=(m, n)), rng.normal(size=(m, n))

    def f(name, val):
        out, x = blk.residual_norm(**{**v, name: val}, scale=0.7, eps=1e-3)
        return (x * dx).sum() + (out * dr).sum()
    out, _ = blk.residual_norm(**v, scale=0.7, eps=1e-3)
    rest = {k: v[k] for k in ("y", "post_w", "gate")}
    g = blk.residual_norm_backward(out, v["pre_w"], dx, dr, **rest, scale=0.7, eps=1e-3)
    for name, grad in (("r", "dr"), ("pre_w", "dpre_weight"), ("y", "dy"), ("post_w", "dpost_weight"),
                       ("gate", "dgate")):
        if v[name] is None:
            assert grad not in g
            continue
        for i in np.ndindex(v[name].shape):
            assert abs(_diff(lambda a: f(name, a), v[name], i, 1e-5) - g[grad][i]) < 1e-7, (name, i)


def test_norm_without_a_block_only_norms():
    r = np.array([[3.0, 4.0]])
    out, x = blk.residual_norm(r, np.array([1.0, 2.0]), eps=0.0)
    assert out is r and np.allclose(x, [[3 / math.sqrt(12.5), 8 / math.sqrt(12.5)]])


def test_sampler_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    ids = lambda **kw: sorted(blk.kept_set(l, **kw)[0].tolist())  # noqa: E731
    assert ids() == [0, 1, 2, 3]
    assert ids(top_k=2) == [1, 3]
    assert ids(top_p=0.5) == [1, 3] and ids(top_p=0.39) == [1] and ids(top_p=0.0) == [1]
    assert ids(min_p=0.6) == [1, 3] and ids(min_p=2.0) == [1]
    assert ids(top_k=3, top_p=0.7) == [1, 3]      # of 0.9: 0.4, 0.7 >= 0.63
    assert ids(temperature=0.0) == [1]
    # index order: 0.1 | 0.5 | 0.7 | 1.0
    for u, tok in ((0.0, 0), (0.05, 0), (0.3, 1), (0.55, 2), (0.75, 3), (1.0, 3), (float("nan"), 0)):
        assert blk.sample(l, u)[0] == tok, u
    assert abs(blk.sample(l, 0.3)[1] - math.log(0.4)) < 1e-12
    assert abs(blk.sample(l, 0.9, top_k=2)[1] - math.log(0.3 / 0.7)) < 1e-12


def test_sampler_masks_and_ties():
    inf = np.inf
    assert blk.sample([-inf, np.nan, -inf], 0.3) == (-1, -inf)
    assert blk.sample([-inf, 2.0, np.nan], 0.99)[0] == 1
    assert blk.sample([1.0, inf, 0.0, inf], 0.6)[0] == 3
    assert blk.kept_set([1.0, 1.0, 1.0, 1.0], top_k=2)[0].tolist() == [0, 1]
    assert blk.kept_set([1.0, 1.0, 1.0, 1.0], top_p=0.5)[0].tolist() == [0, 1]


def test_sampler_against_enumeration():
    # every row entry tested on its own against the three rules
    rng = np.random.default_rng(3)
    for _ in range(200):
        n = int(rng.integers(1, 12))
        l = np.round(rng.normal(size=n) * 2, 1)   # ties happen
        k, p, mp, t = int(rng.integers(0, n + 2)), rng.random() * 1.2, rng.random() * 0.5, 0.3 + rng.random()
        w = np.exp((l - l.max()) / t)
        ahead = lambda i: [j for j in range(n) if l[j] > l[i] or (l[j] == l[i] and j < i)]  # noqa: E731
        first = [i for i in range(n) if not 0 < k < n or len(ahead(i)) < k]
        s = sum(w[i] for i in first)
        want = [i for i in first if w[i] >= mp
                and (p >= 1 or not ahead(i) or sum(w[j] for j in ahead(i)) < p * s - 1e-12
                     or abs(sum(w[j] for j in ahead(i)) - p * s) < 1e-12)]
        got = sorted(blk.kept_set(l, t, k, p, mp)[0].tolist())
        assert got == want

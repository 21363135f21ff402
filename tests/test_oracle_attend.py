"""Pins of the oracle of the attention sublayer and of log probabilities: its
gradients against central differences of its forward formulas, its attention
against a softmax written out for whole sequences, hand-worked rows.  No GPU."""
import math

import numpy as np
import pytest

from oracle import q3_attend as att


def _diff(f, x, i, d=1e-5):
    up, dn = x.copy(), x.copy()
    up[i] += d
    dn[i] -= d
    return (f(up) - f(dn)) / (2 * d)


def test_rotation_by_hand():
    x = np.arange(6.0).reshape(1, 1, 6)
    pos, freq = np.array([1.0]), np.array([math.pi / 2, math.pi])
    half = att.head_norm_rope(x, None, pos, freq, 0.0)
    assert np.allclose(half[0, 0], [-2, -1, 0, -3, 4, 5])      # (0, 2) by a quarter, (1, 3) by a half turn
    pairs = att.head_norm_rope(x, None, pos, freq, 0.0, True)
    assert np.allclose(pairs[0, 0], [-1, 0, -2, -3, 4, 5])
    # scores of rotated heads depend on the distance alone
    rng = np.random.default_rng(0)
    q, k, f = rng.normal(size=(1, 1, 8)), rng.normal(size=(1, 1, 8)), np.array([1.0, 0.3, 0.07, 0.01])
    dot = lambda a, b: float((att.head_norm_rope(q, None, np.array([a]), f, 0.0)  # noqa: E731
                              * att.head_norm_rope(k, None, np.array([b]), f, 0.0)).sum())
    assert abs(dot(100.0, 97.0) - dot(5.0, 2.0)) < 1e-12


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("turned", [0, 2, 6])
def test_rope_gradient(norm, interleaved, turned):
    rng = np.random.default_rng(1)
    x, g = rng.normal(size=(2, 3, 6)), rng.normal(size=(2, 3, 6))
    w = rng.normal(size=6) if norm else None
    pos, freq = np.array([3.0, 70000.0]), rng.random(turned // 2)
    f = lambda a, b: (att.head_norm_rope(a, b, pos, freq, 1e-3, interleaved) * g).sum()  # noqa: E731
    dx, dw = att.head_norm_rope_backward(x, g, w, pos, freq, 1e-3, interleaved)
    for i in np.ndindex(x.shape):
        assert abs(_diff(lambda a: f(a, w), x, i) - dx[i]) < 1e-7
    assert (dw is None) == (not norm)
    for i in range(6 if norm else 0):
        assert abs(_diff(lambda b: f(x, b), w, i) - dw[i]) < 1e-7


def test_paged_attention_is_attention():
    rng = np.random.default_rng(2)
    hq, hk, d, size = 4, 2, 5, 4
    length, new = 11, 3
    keys, values = rng.normal(size=(length, hk, d)), rng.normal(size=(length, hk, d))
    q = rng.normal(size=(new, hq, d))
    table = np.array([[5, 0, 2]])
    k, v = np.full((6, hk, size, d), np.nan), np.full((6, hk, size, d), np.nan)
    for p in range(length):
        k[table[0, p // size], :, p % size], v[table[0, p // size], :, p % size] = keys[p], values[p]
    for window in (0, 1, 2, 7, 50):
        out, lse, _ = att.paged_attention(q, k, v, [0, new], [length], table, 0.7, window)
        for i in range(new):
            p = length - new + i
            first = max(0, p - window + 1) if window else 0
            for h in range(hq):
                e = np.exp(0.7 * keys[first:p + 1, h // 2] @ q[i, h])
                assert np.allclose(out[i, h], e @ values[first:p + 1, h // 2] / e.sum())
                assert abs(lse[i, h] - math.log(e.sum())) < 1e-12


def test_places_and_pages():
    # two tokens at positions 3, 4; none; three at -1, 0, 1; a row of no sequence
    w = att.places([0, 2, 2, 5], [5, 9, 2], 6)
    assert w.tolist() == [[0, 3], [0, 4], [2, -1], [2, 0], [2, 1], [-1, -1]]
    table = np.array([[3, -1, 9]])
    assert att.find(table, 4, 8, 0, 7) == (3, 7) and att.find(table, 4, 8, 0, 8) is None
    assert att.find(table, 4, 8, 0, 16) is None and att.find(table, 10, 8, 0, 16) == (9, 0)
    assert att.find(table, 4, 8, 0, 24) is None and att.find(table, 4, 8, 0, -1) is None


def test_logprobs_by_hand():
    inf, nan = np.inf, np.nan
    lp, h, ids, lps = att.logprobs(np.log([0.1, 0.4, 0.2, 0.3]), 2, 1.0, 3)
    assert abs(lp - math.log(0.2)) < 1e-12 and ids.tolist() == [1, 3, 2]
    assert abs(h + sum(p * math.log(p) for p in (0.1, 0.4, 0.2, 0.3))) < 1e-12
    assert np.allclose(np.exp(lps), [0.4, 0.3, 0.2])
    assert att.logprobs([1.0, 1.0, 1.0], 5, 1.0, 2)[0] == 0.0
    assert att.logprobs([1.0, 1.0, 1.0], 0, 1.0, 2)[2].tolist() == [0, 1]
    lp, h, ids, lps = att.logprobs([-inf, nan, 2.0], 0, 0.5, 2)
    assert lp == -inf and h == 0 and ids.tolist() == [2, -1] and lps.tolist() == [0.0, -inf]
    lp, h, ids, _ = att.logprobs([1.0, inf, 0.0, inf], 3, 1.0, 3)
    assert abs(lp + math.log(2)) < 1e-12 and abs(h - math.log(2)) < 1e-12 and ids.tolist() == [1, 3, 0]
    lp, h, ids, lps = att.logprobs([-inf, nan], 1, 1.0, 1)
    assert lp == -inf and h == 0 and ids.tolist() == [-1] and lps[0] == -inf


@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("target", [-1, 0, 3])
def test_logprobs_gradient(temperature, target):
    rng = np.random.default_rng(3)
    row = rng.normal(size=7) * 2
    f = lambda r: 0.7 * att.logprobs(r, target, temperature)[0] - 1.3 * att.logprobs(r, target, temperature)[1]  # noqa: E731
    d = att.logprobs_backward(row, target, 0.7, -1.3, temperature)
    for i in range(7):
        assert abs(_diff(f, row, (i,)) - d[i]) < 1e-8
    masked = row.copy()
    masked[[2, 3]] = -np.inf, np.nan
    d = att.logprobs_backward(masked, target, 0.7, -1.3, temperature)
    assert d[2] == 0 and d[3] == 0
    live = [0, 1, 4, 5, 6]
    if target != 3:
        rest = att.logprobs_backward(row[live], target, 0.7, -1.3, temperature)
        assert np.allclose(d[live], rest)

"""The oracle of the attention sublayer and of log probabilities (fp64).

Plain formulas on float64 arrays, one token, head and position at a time where
that is what the definition says.  Nothing here rounds: the tests add the
roundings of the result types to their bounds.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ head norms and rotation

def _turn(x, angle, interleaved, sign=1.0):
    """The first 2 len(angle) values of x [..., d] rotated in pairs."""
    h = angle.shape[-1]
    c, s = np.cos(angle), sign * np.sin(angle)
    a, b = (np.arange(h) * 2, np.arange(h) * 2 + 1) if interleaved else (np.arange(h), np.arange(h) + h)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def head_norm_rope(x, weight, positions, freq, eps, interleaved=False):
    """x [m][heads][d] -> its normed (weight given) and rotated heads."""
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    return _turn(x, positions[:, None, None] * freq, interleaved)


def head_norm_rope_backward(x, g, weight, positions, freq, eps, interleaved=False):
    """-> (dx, dweight) for the gradient g of the rotated heads (dweight None without a norm)."""
    dn = _turn(g, positions[:, None, None] * freq, interleaved, -1.0)
    if weight is None:
        return dn, None
    s = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * s
    a = dn * weight
    return s * (a - h * (a * h).mean(-1, keepdims=True)), (dn * h).sum((0, 1))


# ------------------------------------------------------------------ paged batches

def places(q_start, kv_len, m):
    """(sequence, position) of each of m rows; sequence -1: the row belongs to none."""
    out = np.full((m, 2), -1, np.int64)
    for s in range(len(kv_len)):
        for i in range(max(0, q_start[s]), min(m, q_start[s + 1])):
            out[i] = s, kv_len[s] - (q_start[s + 1] - i)
    return out


def find(page_table, pages, page_size, s, p):
    """(page, place) of position p of sequence s, or None where it is not there."""
    if p < 0 or p // page_size >= page_table.shape[1]:
        return None
    page = page_table[s, p // page_size]
    return (int(page), int(p % page_size)) if 0 <= page < pages else None


def paged_attention(q, k, v, q_start, kv_len, page_table, scale, window=0):
    """q [m][hq][d], k and v [pages][heads][page_size][d] -> (out, lse, size): size
    is sum softmax |v|, which bounds what a relative error of the weights does.
    Rows that belong to no sequence are NaN."""
    m, hq, d = q.shape
    pages, heads, page_size, _ = k.shape
    out, size = np.full((m, hq, d), np.nan), np.full((m, hq, d), np.nan)
    lse = np.full((m, hq), np.nan)
    where = places(q_start, kv_len, m)
    for s in range(len(kv_len)):
        rows = np.flatnonzero(where[:, 0] == s)
        if not len(rows):
            continue
        last = int(where[rows, 1].max())
        there = [(p, f) for p in range(last + 1) if (f := find(page_table, pages, page_size, s, p)) is not None]
        at = np.array([p for p, _ in there], np.int64)
        ks = np.array([k[f[0], :, f[1]] for _, f in there]).reshape(len(at), heads, d)
        vs = np.array([v[f[0], :, f[1]] for _, f in there]).reshape(len(at), heads, d)
        for i in rows:
            p = where[i, 1]
            seen = (at <= p) & ((at > p - window) if window else True)
            for h in range(hq):
                g = h // (hq // heads)
                if not seen.any():
                    out[i, h], size[i, h], lse[i, h] = 0, 0, -np.inf
                    continue
                sc = scale * (ks[seen, g] @ q[i, h])
                w = np.exp(sc - sc.max())
                lse[i, h] = sc.max() + np.log(w.sum())
                w /= w.sum()
                out[i, h], size[i, h] = w @ vs[seen, g], w @ np.abs(vs[seen, g])
    return out, lse, size


# ------------------------------------------------------------------ log probabilities

def live_entries(row):
    """Entries that carry weight: neither -inf nor NaN, only +inf where there is one."""
    live = ~np.isnan(row) & (row != -np.inf)
    return live & (row == np.inf) if (row == np.inf).any() else live


def log_softmax(row, temperature=1.0):
    """ln p of a row; -inf where an entry has no weight."""
    row = np.asarray(row, np.float64)
    out, live = np.full(len(row), -np.inf), live_entries(row)
    if live.any():
        top = row[live].max()
        z = np.zeros(live.sum()) if top == np.inf else (row[live] - top) / temperature
        out[live] = z - np.log(np.exp(z).sum())
    return out


def entropy(logp):
    l = logp[logp > -np.inf]
    return float(-(np.exp(l) * l).sum()) if len(l) else 0.0


def logprobs(row, target, temperature=1.0, top=0):
    """-> (logprob, entropy, ids, logprobs of the ids) of one row."""
    logp = log_softmax(row, temperature)
    n = len(row)
    lp = float(logp[target]) if 0 <= target < n else 0.0
    with np.errstate(invalid="ignore"):
        order = [int(i) for i in np.lexsort((np.arange(n), -np.asarray(row, np.float64)))
                 if not np.isnan(row[i]) and row[i] != -np.inf][:top]
    ids = np.array(order + [-1] * (top - len(order)), np.int32)
    return lp, entropy(logp), ids, np.array([logp[i] if i >= 0 else -np.inf for i in ids])


def logprobs_backward(row, target, dlogprob, dentropy, temperature=1.0):
    logp = log_softmax(row, temperature)
    p, h = np.exp(logp), entropy(logp)
    safe = np.where(logp > -np.inf, logp, 0.0)
    d = -dentropy * p * (safe + h)
    if 0 <= target < len(row):
        d -= dlogprob * p
        if logp[target] > -np.inf:
            d[target] += dlogprob
    return d / temperature

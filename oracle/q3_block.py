"""The oracle of the operators between and behind the packed products (fp64).

Plain formulas on float64 arrays; weights come dequantised from
q3_oracle.dequantize.  Nothing here rounds: the tests add the roundings of the
result types to their bounds.
"""
from __future__ import annotations

import numpy as np


def _logistic(v):
    """1 / (1 + e^-v), exact to fp64 at both ends (0.5 (1 + tanh(v/2)) is 0 from
    v = -38 on)."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _inner(name: str, z):
    """v with act(z) = z / (1 + e^-v), and dv/dz: 1/2 (1 + tanh t) = 1 / (1 + e^-2t)."""
    if name == "silu":
        return z, np.ones_like(z)
    c = 2.0 * np.sqrt(2.0 / np.pi)
    return c * (z + 0.044715 * z ** 3), c * (1.0 + 3 * 0.044715 * z * z)


def act(name: str, z):
    """silu(z) = z / (1 + e^-z); gelu: z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))."""
    z = np.asarray(z, np.float64)
    return z * _logistic(_inner(name, z)[0])


def act_slope(name: str, z):
    z = np.asarray(z, np.float64)
    v, dv = _inner(name, z)
    p, q = _logistic(v), _logistic(-v)
    with np.errstate(over="ignore", invalid="ignore"):
        return p + np.where(p * q > 0, z * (p * q) * dv, 0.0)


def glu(w, x, name: str):
    """w [2I][K], x [m][K] -> (h [m][I], pre [m][2I])."""
    pre = x @ w.T
    i = w.shape[0] // 2
    return act(name, pre[:, :i]) * pre[:, i:], pre


def glu_backward(pre, dh, name: str):
    i = pre.shape[1] // 2
    g, u = pre[:, :i], pre[:, i:]
    return np.concatenate([dh * u * act_slope(name, g), dh * act(name, g)], 1)


def _root(v, eps):
    return 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)


def residual_norm(r, pre_w=None, y=None, post_w=None, gate=None, scale=1.0, eps=1e-6):
    """-> (r', x); the weights default to 1."""
    out = r
    if y is not None:
        t = y if post_w is None else y * _root(y, eps) * post_w
        out = r + scale * (1.0 if gate is None else gate) * t
    x = out * _root(out, eps)
    return out, x if pre_w is None else x * pre_w


def residual_norm_backward(out, pre_w=None, dx=None, dr_out=None, y=None, post_w=None, gate=None, scale=1.0,
                           eps=1e-6):
    """Gradients from the kept r', by the chain rule on each row."""
    n = out.shape[1]
    s = _root(out, eps)
    h = out * s
    dx = np.zeros_like(out) if dx is None else dx
    a = dx if pre_w is None else dx * pre_w
    g = s * (a - h * (a * h).sum(1, keepdims=True) / n)
    if dr_out is not None:
        g = g + dr_out
    res = {"dr": g, "dpre_weight": (dx * h).sum(0)}
    if y is None:
        return res
    dt = scale * g * (1.0 if gate is None else gate)
    if post_w is None:
        t, res["dy"] = y, dt
    else:
        sy = _root(y, eps)
        yh = y * sy
        t = yh * post_w
        b = dt * post_w
        res["dpost_weight"] = (dt * yh).sum(0)
        res["dy"] = sy * (b - yh * (b * yh).sum(1, keepdims=True) / n)
    if gate is not None:
        dg = scale * g * t
        res["dgate"] = dg.sum(0) if np.ndim(gate) == 1 else dg
    return res


def kept_set(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(indices ranked, weights) of one row's kept entries, best first."""
    l = np.asarray(logits, np.float64)
    n = len(l)
    live = np.flatnonzero(~np.isnan(l) & (l != -np.inf))
    if len(live) == 0:
        return live, np.zeros(0)
    top = l[live].max()
    if top == np.inf:
        live = live[l[live] == np.inf]
    order = live[np.lexsort((live, -l[live]))]
    greedy = temperature <= 0
    t = 1.0 if greedy or np.isnan(temperature) else float(temperature)
    if greedy:
        return order[:1], np.ones(1)
    with np.errstate(invalid="ignore", under="ignore"):
        w = np.where(l[order] == top, 1.0, np.exp((l[order] - top) / t))
    if 0 < top_k < n:
        order, w = order[:top_k], w[:top_k]
    keep = np.ones(len(order), bool)
    if top_p < 1:
        keep &= (np.cumsum(w) - w < top_p * w.sum()) | (np.arange(len(w)) == 0)
    if min_p > 0:
        keep &= w >= min(float(min_p), 1.0)
    return order[keep], w[keep]


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row's (token, logprob)."""
    order, w = kept_set(logits, temperature, top_k, top_p, min_p)
    if len(order) == 0:
        return -1, -np.inf
    by_index = np.argsort(order)
    order, w = order[by_index], w[by_index]
    u = 0.0 if not u > 0 else float(u)
    run = np.cumsum(w)
    hit = np.flatnonzero((run > u * run[-1]) & (w > 0))
    at = hit[0] if len(hit) else np.flatnonzero(w > 0)[-1]
    return int(order[at]), float(np.log(w[at] / run[-1]))

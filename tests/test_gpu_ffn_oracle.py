"""The feed-forward sublayer with all it can take (post norm, gate, scale, next
norm) against the fp64 oracle, end to end, on the GPU.

The oracle rounds where the definition does, to bf16 behind the first norm and
behind the gated block, and bounds are carried from call to call.  Rounding is
monotone: a value known to within e comes out between the roundings of v - e and
v + e, mostly the same number.  A product of k terms is off by k 2^-23 of the
magnitudes and by what its input is; activations' slopes stay below 1.13 and their
own error below 2^-18.  A norm of v off by e per element: the root mean square (with
eps, a 2-norm) moves by at most d = rms(e), so its inverse by the factor 1 + q at
most, q = d / (rms - d), and v s by s (|v| q + e (1 + q)); fp32 statistics add 2^-17."""
import numpy as np
import pytest
import torch

from oracle import q3_block as blk
from test_gpu_block import Block, gen, h64, q3  # noqa: F401

pytestmark = pytest.mark.gpu
U = 2.0 ** -17
CASES = [(96, 64, 3), (160, 96, 70), (512, 1056, 17), (96, 160, 200)]


def to_bf16(v):
    """Round to nearest even with 8 significant bits (normal numbers)."""
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -120))) - 7)
    return np.rint(v / step) * step


def rounded(v, e):
    """bf16(v), and how far the bf16 of something within e of v may be from it."""
    b = to_bf16(v)
    return b, np.maximum(np.abs(to_bf16(v + e) - b), np.abs(to_bf16(v - e) - b))


def product(x, ex, w):
    aw = np.abs(w.T)
    return x @ w.T, (ex + x.shape[1] * 2.0 ** -23 * (np.abs(x) + ex)) @ aw


def normed(v, e, w, eps):
    """norm(v; w) and how far it is off for v off by e."""
    size = np.sqrt((v * v).mean(1, keepdims=True) + eps)
    d = np.sqrt((e * e).mean(1, keepdims=True))
    assert (d < size / 2).all()
    q = d / (size - d)
    t = v / size * w
    off = np.abs(w) / size * (np.abs(v) * q + e * (1 + q))
    return t, off + U * (np.abs(t) + off)


def sublayer(b, r, gate, scale, eps, act):
    """(r', its bound, x, its bound, the block's term before gate and scale) in fp64, r' unrounded."""
    x, ex = rounded(*normed(r, np.zeros_like(r), b.pre64, eps))
    pre, e = product(x, ex, b.gu64)
    i = b.inter
    g, u, eg, eu = pre[:, :i], pre[:, i:], e[:, :i], e[:, i:]
    a = blk.act(act, g)
    eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu
    h = a * u
    h, eh = rounded(h, eh + 2.0 ** -18 * (np.abs(h) + eh))
    t, et = normed(*product(h, eh, b.dn64), b.post64, eps)
    f = scale * gate
    out = r + f * t
    eo = np.abs(f) * et + 2.0 ** -22 * (np.abs(r) + np.abs(f) * (np.abs(t) + et))
    nxt, en = rounded(*normed(out, eo, b.next64, eps))
    return out, eo, nxt, en, t


@pytest.mark.parametrize("k,inter,m", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act,gated", [("silu", "full"), ("gelu", "row"), ("silu", None)])
def test_whole_sublayer(q3, k, inter, m, dtype, act, gated):  # noqa: F811
    b = Block(q3, k, inter, seed=3)
    b.pre64, b.post64, b.next64 = h64(b.pre), h64(b.post), h64(b.next)
    r = gen(m, k, seed=1).to(dtype)
    gate = {"full": gen(m, k, seed=5), "row": gen(k, seed=5), None: None}[gated]
    scale, eps = 0.75, 1e-5
    got_r, got_x = (h64(t) for t in q3.q3_ffn(b.gu, b.dn, r, b.pre, b.post, gate, scale, b.next, act=act, eps=eps))
    out, eo, nxt, en, t = sublayer(b, h64(r), 1.0 if gate is None else h64(gate), scale, eps, act)
    # what the bounds tell from the right answer: no term, no gate, no scale
    for other in (h64(r), h64(r) + t * (1.0 if gate is None else h64(gate))) + ((h64(r) + scale * t,) if gated else ()):
        assert (np.abs(other - out) > 4 * eo).mean() > 0.2
    if dtype == torch.bfloat16:
        out, eo = rounded(out, eo)
    assert (np.abs(got_r - out) <= eo).all()
    assert (np.abs(got_x - nxt) <= en).all()

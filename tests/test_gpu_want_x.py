"""q3_residual_norm and q3_ffn without the norm of r': r' is bitwise what it is with it."""
import pytest
import torch

from test_gpu_block import Block, gen, q3  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n", [(1, 4096), (3, 100), (70, 513), (2, 9000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_residual_norm(q3, m, n, dtype):  # noqa: F811
    r, y, w, gate = gen(m, n, seed=1).to(dtype), gen(m, n, seed=2), gen(n, seed=3, base=1.0), gen(n, seed=4)
    want, _ = q3.q3_residual_norm(r, w, y, w, gate, 0.5)
    got, x = q3.q3_residual_norm(r, None, y, w, gate, 0.5, want_x=False)
    assert x is None and torch.equal(got, want)
    own = r.clone()
    got, x = q3.q3_residual_norm(own, None, y, w, gate, 0.5, r_out=own, want_x=False)
    assert got is own and x is None and torch.equal(own, want)
    copy, x = q3.q3_residual_norm(r, r_out=torch.empty_like(r), want_x=False)
    assert x is None and torch.equal(copy, r)
    for bad in (dict(pre_weight=w), dict(x=torch.empty(m, n, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            q3.q3_residual_norm(r, y=y, want_x=False, **bad)
    with pytest.raises(ValueError):
        q3.q3_residual_norm(r, want_x=False)


@pytest.mark.parametrize("m", [1, 17, 70, 150])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ffn(q3, m, dtype):  # noqa: F811
    b = Block(q3, 96, 160)
    r = gen(m, 96, seed=9).to(dtype)
    want, _ = q3.q3_ffn(b.gu, b.dn, r, b.pre, b.post, None, 0.5, b.next)
    got, x = q3.q3_ffn(b.gu, b.dn, r, b.pre, b.post, None, 0.5, want_x=False)
    assert x is None and torch.equal(got, want)
    own = r.clone()
    q3.q3_ffn(b.gu, b.dn, own, b.pre, b.post, None, 0.5, r_out=own, want_x=False)
    assert torch.equal(own, want)
    for bad in (dict(next_weight=b.next), dict(x=torch.empty(m, 96, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            q3.q3_ffn(b.gu, b.dn, r, b.pre, want_x=False, **bad)


def test_decode_loop_as_documented(q3):  # noqa: F811
    blocks = [Block(q3, 96, 64, seed=s) for s in (0, 10, 20)]
    r = gen(5, 96, seed=1).to(torch.bfloat16)
    a = b = r
    for i, l in enumerate(blocks):
        a, xa = q3.q3_ffn(l.gu, l.dn, a, l.pre, next_weight=l.next)
        last = i == len(blocks) - 1
        b, xb = q3.q3_ffn(l.gu, l.dn, b, l.pre, next_weight=l.next if last else None, want_x=last)
    assert torch.equal(a, b) and torch.equal(xa, xb)

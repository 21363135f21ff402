"""Equal calls give equal bits, whatever ran between them: every operator of
include/q3_block.h at ragged sizes of each of its forms."""
import pytest
import torch

import synth
from gpu_util import pack_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def rand(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda().to(dtype)


def flat(v):
    if v is None or isinstance(v, torch.Tensor):
        return [] if v is None else [v]
    return [t for x in (vars(v).values() if hasattr(v, "__dict__") else v) for t in flat(x)]


def same(call, other):
    first = [t.clone() for t in flat(call())]
    for _ in range(4):
        other()
        again = flat(call())
        assert len(first) == len(again)
        for a, b in zip(first, again):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n,k,m", [(64, 192, 1), (1408, 4384, 3), (832, 544, 46), (704, 1024, 65), (512, 2048, 128),
                                   (9472, 160, 130), (256, 4128, 100), (2048, 1536, 1700), (6016, 64, 17)])
def test_products_and_gated_block(q3, n, k, m):
    w = pack_layer(q3, synth.make_layer(n, k, seed=n))
    x, x2 = (rand(m, k, seed=s, dtype=torch.bfloat16) for s in (1, 2))
    dy, dy2 = (rand(m, n, seed=s, dtype=torch.bfloat16) for s in (3, 4))
    dh = rand(m, n // 2, seed=5)
    same(lambda: q3.q3_gemm(w, x), lambda: q3.q3_gemm(w, x2))
    same(lambda: q3.q3_gemm_backward(w, dy), lambda: q3.q3_gemm_backward(w, dy2))
    for act in ("silu", "gelu"):
        def step(a):
            h, pre = q3.q3_glu(w, a, act=act, save_pre=True)
            return h, pre, q3.q3_glu_backward(pre, dh, act=act)
        same(lambda: step(x), lambda: step(x2))


@pytest.mark.parametrize("m,n", [(1, 4096), (1379, 1276), (139, 453), (41, 9012), (600, 12288), (30, 16000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norms(q3, m, n, dtype):
    r, y, dx = rand(m, n, seed=1, dtype=dtype), rand(m, n, seed=2), rand(m, n, seed=3)
    w, gate = rand(n, seed=4), rand(n, seed=5)

    def forward(v):
        return q3.q3_residual_norm(r, w, v, w, gate, 0.5)

    def back(v):
        return q3.q3_residual_norm_backward(r, w, v, r, y, w, gate, 0.5)
    same(lambda: forward(y), lambda: forward(dx))
    same(lambda: back(dx), lambda: back(y))


@pytest.mark.parametrize("m,n", [(1, 188), (69, 5517), (18, 37125), (3, 151936)])
def test_sampling(q3, m, n):
    l, l2 = rand(m, n, seed=1), rand(m, n, seed=2) * 3
    u = torch.rand(m, generator=torch.Generator().manual_seed(3)).cuda()
    k, p = torch.full((m,), 60, dtype=torch.int32, device="cuda"), torch.full((m,), 0.9, device="cuda")
    for kw in (dict(), dict(top_k=k, top_p=p), dict(top_p=p, temperature=p / 9)):
        same(lambda: q3.q3_sample(l, u, **kw), lambda: q3.q3_sample(l2, u, **kw))

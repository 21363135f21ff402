"""One token's NaN or infinity stays its own in the expert passes and the draft
head's scores too, where K ends inside a 512-column step (lanes without groups
there have the next token's row in their place)."""
import pytest
import torch

import synth
from gpu_util import dev, pack_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def stack(q3, count, n, k, seed):
    st = q3.empty_stack(count, n, k, "cuda")
    for e in range(count):
        layer = synth.make_layer(n, k, seed=seed + e)
        q3.q3_pack(dev(layer.codes), dev(layer.scales), dev(layer.codebook), out=st.expert(e))
    return st


def others_keep(call, x, clean):
    for bad in range(x.shape[0]):
        for value in (float("nan"), float("inf")):
            y = x.clone()
            y[bad] = value
            got = call(y)
            rows = [i for i in range(x.shape[0]) if i != bad]
            assert torch.equal(got[rows], clean[rows]), (bad, value)
            assert not torch.isfinite(got[bad]).all()


# whole steps, one quad, two and three quads in the last step, groups that end inside a quad
KS = [512, 96, 544, 800, 928, 1376, 2112]


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("t,topk", [(2, 1), (5, 2), (8, 2)])
def test_expert_passes(q3, k, t, topk):
    count, inter = 5, 160
    x = torch.randn(t, k, generator=torch.Generator().manual_seed(k)).cuda().to(torch.bfloat16)
    logits = torch.randn(t, count, generator=torch.Generator().manual_seed(t)).cuda()
    ids = q3.q3_moe_topk(logits, topk)
    st = stack(q3, count, 2 * inter, k, 1)
    call = lambda a: q3.q3_grouped_expert_gemv(st, a, ids, False).view(t, topk, -1)  # noqa: E731
    others_keep(call, x, call(x))
    dn = stack(q3, count, 96, inter, 50)          # its K, 160, ends inside a step as well
    mlp = lambda a: q3.q3_moe_mlp(st, dn, a, ids, logits)  # noqa: E731
    others_keep(mlp, x, mlp(x))


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("m", [2, 7, 16])
def test_head_scores(q3, k, m):
    head, x = synth.make_head(100, k, m, seed=k + m)
    w2 = q3.q3_pack2(dev(head.codes), dev(head.scales), dev(head.codebook))
    call = lambda a: q3.q3_head2_scores(w2, a)  # noqa: E731
    a = dev(x).view(torch.bfloat16)
    others_keep(call, a, call(a))


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("n", [48, 9000])
def test_small_products(q3, n, k):
    w = pack_layer(q3, synth.make_layer(n, k, seed=k))
    for m, calls in ((3, (q3.q3_gemv, q3.q3_gemm_small_m)), (8, (q3.q3_gemv, q3.q3_gemm_small_m)),
                     (13, (q3.q3_gemm_small_m,)), (29, (q3.q3_gemm_small_m,)), (48, (q3.q3_gemm_small_m,))):
        x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).cuda().to(torch.bfloat16)
        for f in calls:
            others_keep(lambda a: f(w, a), x, f(w, x))

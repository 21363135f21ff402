"""Residual norms of more rows than one launch takes threads for (2^26 - 4 up to
512 columns, 2^22 - 1 past 4096): the rows on both sides of the border and the
last ones as they come out alone, on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def sample(most, m):
    return torch.tensor([0, 1, most - 2, most - 1, most, most + 1, m - 1], device="cuda")


@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("gate", ["full", "row"])
def test_short_rows(q3, n, gate):
    most = (1 << 26) - 4
    m = most + 9
    g = torch.Generator(device="cuda").manual_seed(n)
    r, y, gt = (torch.randn(m, n, generator=g, device="cuda") for _ in range(3))
    if gate == "row":
        gt = gt[0].contiguous()
    w = torch.rand(n, generator=g, device="cuda") + 0.5
    r1, x = q3.q3_residual_norm(r, w, y, w, gt, 0.5)
    at = sample(most, m)
    r2, x2 = q3.q3_residual_norm(r[at], w, y[at], w, gt[at] if gate == "full" else gt, 0.5)
    assert torch.equal(r1[at], r2) and torch.equal(x[at], x2)
    del r1, x
    q3.q3_residual_norm(r, w, y, w, gt, 0.5, r_out=r)
    assert torch.equal(r[at], r2)


def test_long_rows(q3):
    most, n = (1 << 22) - 1, 4104
    m = most + 6
    r = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")   # 34 GB
    r.copy_(torch.randn(n, device="cuda"))
    at = sample(most, m)
    r[at] = torch.randn(len(at), n, device="cuda").to(torch.bfloat16)
    w = torch.rand(n, device="cuda") + 0.5
    _, x = q3.q3_residual_norm(r, w)
    _, x2 = q3.q3_residual_norm(r[at], w)
    assert torch.equal(x[at], x2)

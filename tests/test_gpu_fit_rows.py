"""Codebook fitting of more rows than one launch takes threads for (2^24 - 1): the
rows on both sides of the border and the last ones as they come out alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_rows_past_one_launch():
    import bit_fp8_codebook_amd as q3
    q3.lib()
    most, k = (1 << 24) - 1, 32
    n = most + 9
    w = torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    at = torch.tensor([0, 1, most - 2, most - 1, most, most + 1, n - 1], device="cuda")
    book = torch.full((n, 8), 0x7F, dtype=torch.uint8, device="cuda")   # NaN: no fitted entry is
    q3.q3_fit_codebook(w, book)
    assert torch.equal(book[at], q3.q3_fit_codebook(w[at].contiguous()))
    assert not (book == 0x7F).any()

"""q3_paged_attention at the ends of its tables, lengths and windows."""
import numpy as np
import pytest
import torch

from paged_util import Paged, cuda
from test_gpu_attend import FORMS, _q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("window", [1, 63, 64, 127, 4096])
@pytest.mark.parametrize("length", [BIG, BIG - 63, BIG - 127, BIG - 4095, BIG - 4200, 2 ** 30])
@pytest.mark.parametrize("form", FORMS)
def test_windows_far_behind_the_table_see_nothing(q3, form, length, window):
    new, hq, hk = form
    p = Paged(np.random.default_rng(21), [new, 1], [new + 30, 20], hk, 64, 16, stale=float("nan"))
    cache, _ = p.on_device(q3)
    q = _q(np.random.default_rng(22), p.m, hq, 64)
    out, lse = torch.full_like(q, 2.0), torch.full((p.m, hq), 2.0, device="cuda")
    far = cuda(np.array([length, length], np.int32))
    q3.q3_paged_attention(q, cache, q3.PagedBatch(cuda(p.start), far, cuda(p.table)), window=window, out=out, lse=lse)
    assert not out.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("form", FORMS)
def test_far_tokens_without_a_window_see_the_whole_table(q3, form):
    new, hq, hk = form
    p = Paged(np.random.default_rng(23), [new, 1], [160, 160], hk, 64, 16)
    cache, _ = p.on_device(q3)
    q = _q(np.random.default_rng(24), p.m, hq, 64)

    def run(length, window):
        batch = q3.PagedBatch(cuda(p.start), cuda(np.array([length, length], np.int32)), cuda(p.table))
        return q3.q3_paged_attention(q, cache, batch, window=window, want_lse=True)
    near = run(160 + new, 0)     # the table ends in front of every new token
    for length, window in ((2 ** 30, 0), (BIG, 0), (BIG, BIG), (BIG - 4200, BIG - 4200)):
        far = run(length, window)
        assert torch.equal(near[0], far[0]) and torch.equal(near[1], far[1]), (length, window)


@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("extra", [32, 200])
@pytest.mark.parametrize("form", FORMS)
def test_nan_reaches_the_lse_of_the_rows_that_see_it(q3, form, extra, d):
    # a NaN score makes the sum NaN; -inf is the lse of rows that see nothing, and no other
    new, hq, hk = form
    length = new + extra
    p = Paged(np.random.default_rng(25), [new, 1], [length, 40], hk, d, 16)
    q = _q(np.random.default_rng(26), p.m, hq, d)

    def run(q):
        cache, batch = p.on_device(q3)
        return q3.q3_paged_attention(q, cache, batch, want_lse=True)
    x = run(q)
    dirty = q.clone()
    dirty[new - 1, d * (hq - 1) + 3] = float("nan")
    y = run(dirty)
    keep = torch.ones(p.m, hq, dtype=torch.bool, device="cuda")
    keep[new - 1, hq - 1] = False
    assert torch.equal(x[1][keep], y[1][keep]) and torch.isnan(y[1][~keep]).all()
    assert torch.isnan(y[0].view(p.m, hq, d)[~keep]).all()
    # one position's key: alone in its wave's tiles at 32 of 33, first, and last of all
    for at in {0, min(32, length - 1), length - 1}:
        page, place = int(p.table[0, at // 16]), at % 16
        was = p.k[page, :, place, 5].clone()
        p.k[page, :, place, 5] = float("nan")
        y = run(q)
        p.k[page, :, place, 5] = was
        sees = torch.zeros(p.m, dtype=torch.bool, device="cuda")
        sees[:new] = torch.arange(length - new, length, device="cuda") >= at
        assert torch.isnan(y[1][sees]).all() and torch.isnan(y[0][sees]).all(), at
        assert torch.equal(x[1][~sees], y[1][~sees]) and torch.equal(x[0][~sees], y[0][~sees]), at


@pytest.mark.parametrize("form", FORMS)
def test_scales_up_to_the_largest(q3, form):
    # scale log2(e) has to be finite: the largest such scale gives zero scores their mean, the next is refused
    new, hq, hk = form
    p = Paged(np.random.default_rng(27), [new], [new + 40], hk, 64, 16)
    cache, batch = p.on_device(q3)
    q = torch.zeros(new, hq * 64, dtype=torch.bfloat16, device="cuda")
    log2e = np.float32(1.4426950408889634)
    scale = np.finfo(np.float32).max / log2e
    with np.errstate(over="ignore"):
        while np.isfinite(np.nextafter(scale, np.float32(np.inf)) * log2e):
            scale = np.nextafter(scale, np.float32(np.inf))
        while not np.isfinite(scale * log2e):
            scale = np.nextafter(scale, np.float32(0))
    want = q3.q3_paged_attention(q, cache, batch, 1.0, want_lse=True)
    for s in (float(scale), -float(scale)):
        got = q3.q3_paged_attention(q, cache, batch, s, want_lse=True)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]), s
    above = float(np.nextafter(scale, np.float32(np.inf)))
    for s in (above, -above, float(np.finfo(np.float32).max)):
        with pytest.raises(q3.Q3Error):
            q3.q3_paged_attention(q, cache, batch, s)


@pytest.mark.parametrize("form", FORMS)
def test_a_table_that_claims_more_pages_than_positions(q3, form):
    # table_pages up to ld_table, whatever that is: 2^60 pages of 16 are more positions than 64 bits hold
    from bit_fp8_codebook_amd import _block
    new, hq, hk = form
    p = Paged(np.random.default_rng(28), [new], [new + 70], hk, 64, 16)
    cache, batch = p.on_device(q3)
    q = _q(np.random.default_rng(29), new, hq, 64)
    want = q3.q3_paged_attention(q, cache, batch, want_lse=True)
    batch._desc = _block.Q3PagedBatch(1, batch.q_start.data_ptr(), batch.kv_len.data_ptr(), batch.page_table.data_ptr(),
                                      1 << 60, 1 << 60)
    got = q3.q3_paged_attention(q, cache, batch, want_lse=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])

"""q3_paged_attention against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import q3_attend as att
from paged_util import BF, F32, Paged, cuda, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


def _run(q3, p, q, scale, window, **kw):
    cache, batch = p.on_device(q3)
    return q3.q3_paged_attention(q, cache, batch, scale, window, want_lse=True, **kw)


def _oracle(p, q, scale, window):
    m = q.shape[0]
    return att.paged_attention(host(q).reshape(m, -1, p.dim), host(p.k), host(p.v), p.start, p.length, p.table, scale,
                               window)


def _check(p, q, out, lse, scale, window):
    """Bounds.  A score is a sum of dim exact products in fp32 and two products more:
    off by (dim + 2) 2^-24 of scale sum |q k|; the weight e^S then by as much,
    relative, and two roundings and an exponential good to 2.  Weights enter the
    second product rounded to bf16; its fp32 sum has one rounding per key; each
    rescaling one (a step of 32 keys or more).  The result is rounded once."""
    m = q.shape[0]
    ref, rl, size = _oracle(p, q, scale, window)
    live = ~np.isnan(rl)
    got, gl = host(out).reshape(ref.shape), host(lse)
    biggest = max(p.length + [1])
    kmax = np.nanmax(np.where(np.isfinite(host(p.k)), np.abs(host(p.k)), 0))
    score = (p.dim + 4) * F32 * abs(scale) * kmax * np.abs(host(q)).reshape(m, -1, p.dim).sum(-1)
    bound = BF * np.abs(ref) + (BF + 2 * biggest * F32 + 8 * F32 + 2 * score[..., None]) * size + 1e-38
    bad = live[..., None] & ~(np.abs(got - ref) <= 1.01 * bound)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], bound[bad][:4])
    empty = live & (rl == -np.inf)
    assert (gl[empty] == -np.inf).all() and (got[empty] == 0).all()
    some = live & ~empty
    off = score[some] + F32 * (biggest + 16 + 2 * np.abs(rl[some]))
    assert (np.abs(gl[some] - rl[some]) <= 1.01 * off).all(), np.abs(gl[some] - rl[some]).max()


def _q(rng, m, hq, d, size=1.5):
    return cuda((size * rng.normal(size=(m, hq * d))).astype(np.float32), torch.bfloat16)


CASES = [  # new, length, hq, hk, d, page, window
    ([1], [1], 1, 1, 64, 16, 0), ([1], [31], 4, 1, 128, 16, 0), ([1], [700], 32, 8, 128, 64, 0),
    ([1] * 5, [3, 64, 65, 1, 300], 8, 2, 128, 16, 0), ([1] * 3, [129, 1000, 32], 3, 3, 256, 32, 0),
    ([1, 1], [2000, 40], 16, 1, 64, 256, 100), ([8, 8], [100, 8], 8, 8, 80, 16, 0), ([5], [777], 64, 8, 128, 64, 0),
    ([4, 0, 7, 1], [300, 9, 7, 65], 12, 4, 96, 8, 0), ([100], [100], 4, 4, 128, 16, 0),
    ([130, 1, 1], [400, 77, 256], 6, 2, 64, 32, 50), ([257], [300], 5, 1, 112, 4, 0), ([64, 3], [64, 500], 7, 1, 192, 1, 0),
    ([33], [161], 2, 2, 16, 2, 33), ([40], [40], 16, 2, 256, 1024, 1), ([300], [1500], 2, 1, 128, 128, 0),
    ([200], [900], 3, 1, 48, 16, 64), ([1] * 70, [(37 * i) % 90 + 1 for i in range(70)], 2, 1, 32, 16, 0),
]


@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(q3, case):
    new, length, hq, hk, d, page, window = case
    rng = np.random.default_rng(len(length) + d + page)
    p = Paged(rng, new, length, hk, d, page)
    q = _q(rng, p.m, hq, d)
    out, lse = _run(q3, p, q, d ** -0.5, window)
    _check(p, q, out, lse, d ** -0.5, window)


@pytest.mark.parametrize("scale", [1.0, -0.3, 1e-3, 40.0])
@pytest.mark.parametrize("new", [1, 9, 140])
def test_scales(q3, scale, new):
    rng = np.random.default_rng(new)
    p = Paged(rng, [new], [new + 150], 2, 64, 16)
    q = _q(rng, p.m, 6, 64, 0.25)
    out, lse = _run(q3, p, q, scale, 0)
    _check(p, q, out, lse, scale, 0)


FORMS = [(1, 4, 1), (6, 4, 1), (6, 16, 1), (12, 4, 1), (20, 4, 1), (50, 8, 2), (130, 2, 1), (70, 6, 2)]   # new, hq, hk: rows of each kernel form


@pytest.mark.parametrize("d", [64, 128, 240, 256])
@pytest.mark.parametrize("form", FORMS)
def test_stale_values_reach_nothing(q3, form, d):
    # infinities and NaN in the cache wherever no sequence stands, and between the pages
    new, hq, hk = form
    for stale in (float("nan"), float("inf"), -float("inf")):
        a, b = (Paged(np.random.default_rng(5), [new, 1], [new + 77, 40], hk, d, 16, stale=s, gap=8) for s in (0.0, stale))
        q = _q(np.random.default_rng(6), a.m, hq, d)
        x, y = _run(q3, a, q, 0.1, 0), _run(q3, b, q, 0.1, 0)
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]), stale


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("form", FORMS)
def test_a_tokens_values_stay_unseen(q3, form, window, bad):
    # one position's key and value are not finite: rows that do not see it are as they were, rows that do are not finite
    new, hq, hk = form
    d, length = 64, new + 75
    for at in (length - 1, length - max(1, new // 2), 60):
        a, b = (Paged(np.random.default_rng(7), [new], [length], hk, d, 8) for _ in range(2))
        page, place = a.table[0, at // 8], at % 8
        b.v[page, :, place, 3] = bad
        q = _q(np.random.default_rng(8), new, hq, d)
        x, y = _run(q3, a, q, 0.1, window), _run(q3, b, q, 0.1, window)
        sees = np.array([at <= p and (not window or at > p - window) for p in range(length - new, length)])
        hid = torch.from_numpy(~sees).cuda()
        assert torch.equal(x[0][hid], y[0][hid]) and torch.equal(x[1], y[1])
        if sees.any():
            seen = y[0][~hid].view(-1, hq, d).float()
            assert not torch.isfinite(seen[:, :, 3]).any()
            keep = [i for i in range(d) if i != 3]
            assert torch.equal(seen[:, :, keep], x[0][~hid].view(-1, hq, d).float()[:, :, keep])
            if bad == float("inf"):
                assert (seen[:, :, 3] == bad).all()
        b.v[page, :, place, 3] = a.v[page, :, place, 3]
        b.k[page, :, place, 2] = bad
        y = _run(q3, b, q, 0.1, window)
        assert torch.equal(x[0][hid], y[0][hid]) and torch.equal(x[1][hid], y[1][hid])


@pytest.mark.parametrize("form", FORMS)
def test_one_query_stays_its_own(q3, form):
    new, hq, hk = form
    p = Paged(np.random.default_rng(9), [new, 2], [new + 200, 50], hk, 128, 16)
    q = _q(np.random.default_rng(10), p.m, hq, 128)
    x = _run(q3, p, q, 0.1, 0)
    dirty = q.clone()
    dirty[0, 128 * (hq - 1) + 3] = float("nan")
    y = _run(q3, p, dirty, 0.1, 0)
    keep = torch.ones(p.m, hq, dtype=torch.bool, device="cuda")
    keep[0, hq - 1] = False
    assert torch.equal(x[0].view(p.m, hq, 128)[keep], y[0].view(p.m, hq, 128)[keep]) and torch.equal(x[1][keep], y[1][keep])
    assert torch.isnan(y[0].view(p.m, hq, 128)[~keep]).all()


@pytest.mark.parametrize("form", FORMS)
def test_rows_without_keys_and_rows_of_no_sequence(q3, form):
    new, hq, hk = form
    rng = np.random.default_rng(11)
    # shorter than its new tokens; nothing at all; an ordinary one; three rows behind the last
    p = Paged(rng, [new, 3, 2], [max(0, new - 3), 0, 30], hk, 64, 16)
    q = _q(rng, p.m + 3, hq, 64)
    out = torch.full_like(q, 3.0)
    lse = torch.full((p.m + 3, hq), 5.0, device="cuda")
    _run(q3, p, q, 0.2, 0, out=out, lse=lse)
    assert (out[p.m:] == 3).all() and (lse[p.m:] == 5).all()
    _check(p, q[:p.m], out[:p.m], lse[:p.m], 0.2, 0)
    assert (lse[:min(3, new)] == -np.inf).all() and (out[new:new + 3] == 0).all()


@pytest.mark.parametrize("form", FORMS)
def test_absent_pages_are_not_seen(q3, form):
    new, hq, hk = form
    rng = np.random.default_rng(12)
    p = Paged(rng, [new, 1], [new + 300, 90], hk, 64, 16)
    pages = p.k.shape[0]
    for entry, at in ((-1, 2), (pages, 5), (2 ** 31 - 1, 0), (-2 ** 31, 7)):
        p.table[0, at] = entry
    p.table[1, :] = [-1] * p.table.shape[1]      # the whole of the second
    q = _q(rng, p.m, hq, 64)
    out, lse = _run(q3, p, q, 0.2, 0)
    _check(p, q, out, lse, 0.2, 0)
    assert (out[-1] == 0).all() and (lse[-1] == -np.inf).all()
    # a table that ends before the sequence does
    p.table = p.table[:, :4].copy()
    out, lse = _run(q3, p, q, 0.2, 0)
    _check(p, q, out, lse, 0.2, 0)


@pytest.mark.parametrize("form", FORMS)
def test_broken_batches_end(q3, form):
    # tables of no sense: the call ends, and rows it does not give to a sequence stay
    new, hq, hk = form
    rng = np.random.default_rng(13)
    p = Paged(rng, [new, 1, 2], [new + 30, 20, 9], hk, 64, 16)
    cache, _ = p.on_device(q3)
    q = _q(rng, p.m, hq, 64)
    big = 2 ** 31 - 1
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    for start, length in ((i32(0, big, big, big), i32(50, 50, 50)), (i32(big, 0, -big, 5), i32(50, 50, 50)),
                          (i32(-7, -3, 4, 2), i32(9, 9, 9)), (i32(0, 1, 2, 3), i32(big, -big, big)),
                          (i32(5, 4, 3, 2), i32(10, 10, 10)), (i32(0, 0, 0, 0), i32(10, 10, 10))):
        out = torch.full_like(q, 2.0)
        q3.q3_paged_attention(q, cache, q3.PagedBatch(start, length, cuda(p.table)), out=out)
        torch.cuda.synchronize()
    assert (out == 2).all()   # the last batch has no rows


@pytest.mark.parametrize("form", FORMS)
def test_equal_calls_give_equal_bits_with_pitched_rows(q3, form):
    new, hq, hk = form
    rng = np.random.default_rng(14)
    p = Paged(rng, [new] * 3, [new + 500, new + 3, new + 1200], hk, 128, 32, wide=3)
    cache, batch = p.on_device(q3)
    q = _q(rng, p.m, hq, 128)
    a, la = q3.q3_paged_attention(q, cache, batch, want_lse=True)
    wide = torch.full((p.m, hq * 128 + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, :-8] = q
    out = torch.full_like(wide, 6.0)
    table = torch.full((3, p.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    table[:, :p.table.shape[1]] = cuda(p.table)
    apart = q3.PagedBatch(batch.q_start, batch.kv_len, table[:, :p.table.shape[1]])
    ws = torch.full((q3.q3_paged_attention_workspace_bytes(p.m, 3, hq, hk, 128) + 256,), 255, dtype=torch.uint8,
                    device="cuda")
    got = q3.q3_paged_attention(wide[:, :-8], cache, apart, out=out[:, :-8], workspace=ws)
    assert torch.equal(out[:, :-8], a) and (out[:, -8:] == 6).all() and got.data_ptr() == out.data_ptr()
    b, lb = q3.q3_paged_attention(q, cache, batch, want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("new", [1, 200])
def test_a_cache_past_32_bits(q3, new):
    # pages 2 GiB apart: offsets of 4 and 6 GiB
    d, hk, page = 64, 1, 64
    rng = np.random.default_rng(15)
    p = Paged(rng, [new], [250], hk, d, page, spare=0)
    pages, stride = p.k.shape[0], 1 << 30
    flat = [torch.empty((pages - 1) * stride + page * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    views = [f.as_strided((pages, hk, page, d), (stride, page * d, d, 1)) for f in flat]
    views[0].copy_(p.k.cuda())
    views[1].copy_(p.v.cuda())
    q = _q(rng, new, 4, d)
    batch = q3.PagedBatch(cuda(p.start), cuda(np.array(p.length, np.int32)), cuda(p.table))
    out, lse = q3.q3_paged_attention(q, q3.PagedCache(*views), batch, want_lse=True)
    _check(p, q, out, lse, d ** -0.5, 0)


def test_long_contexts(q3):
    # one decoded token of 70001 positions beside short ones; verify rows; against torch in fp64
    d, hk, hq, page = 128, 2, 8, 16
    for new in ([1, 1, 1], [9, 2, 5], [100, 1, 1]):
        length = [70001, 130, 2500]
        rng = np.random.default_rng(16)
        p = Paged(rng, new, length, hk, d, page)
        q = _q(rng, p.m, hq, d)
        out, lse = _run(q3, p, q, d ** -0.5, 0)
        kd, vd = p.k.cuda().double(), p.v.cuda().double()
        for s in range(3):
            ids = cuda(p.table[s, :(length[s] + page - 1) // page]).long()
            for h in range(hk):
                k = kd[ids, h].reshape(-1, d)[:length[s]]
                v = vd[ids, h].reshape(-1, d)[:length[s]]
                rows = slice(int(p.start[s]), int(p.start[s + 1]))
                qq = q[rows].view(-1, hq, d)[:, h * 4:h * 4 + 4].double()
                sc = (qq.reshape(-1, d) @ k.t()).view(new[s], 4, -1) * d ** -0.5
                pos = torch.arange(length[s] - new[s], length[s], device="cuda").view(-1, 1, 1)
                sc = sc.masked_fill(torch.arange(length[s], device="cuda") > pos, -float("inf"))
                w = torch.softmax(sc, -1)
                ref, size = (w.view(-1, length[s]) @ v), (w.view(-1, length[s]) @ v.abs())
                got = out[rows].view(-1, hq, d)[:, h * 4:h * 4 + 4].double().reshape(-1, d)
                # scores below 60 in size: their 130 roundings are 5e-4 relative; 70001 keys 2^-24 each
                bound = BF * ref.abs() + (BF + 2 * 70001 * F32 + 1e-3) * size
                assert ((got - ref).abs() <= bound).all()
                ll = torch.logsumexp(sc, -1)
                off = (lse[rows][:, h * 4:h * 4 + 4].double() - ll).abs()
                assert (off <= 1e-3 + 70001 * F32).all()


@pytest.mark.parametrize("d", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("new,length,hq,hk", [
    ([1], [20000], 3, 1), ([20, 1], [20000, 9000], 3, 1), ([400], [800], 48, 24), ([200, 3], [3000, 40], 2, 1)])
def test_many_and_few_parts(q3, new, length, hq, hk, d):
    # tiles in more parts than blocks read at a time, and in a few
    rng = np.random.default_rng(17)
    p = Paged(rng, new, length, hk, d, 64)
    q = _q(rng, p.m, hq, d)
    out, lse = _run(q3, p, q, d ** -0.5, 0)
    _check(p, q, out, lse, d ** -0.5, 0)
    out2, lse2 = _run(q3, p, q, d ** -0.5, 700)
    _check(p, q, out2, lse2, d ** -0.5, 700)


@pytest.mark.parametrize("d", [64, 112, 256])
@pytest.mark.parametrize("new,length", [([300], [500]), ([150, 1, 0, 151], [460, 77, 30, 151])])
@pytest.mark.parametrize("hk", [1, 2, 4])
def test_heads_that_xcds_share(q3, hk, new, length, d):
    # fewer kv heads than XCDs and many tiles, in parts
    rng = np.random.default_rng(18)
    p = Paged(rng, new, length, hk, d, 32)
    q = _q(rng, p.m, 32, d)
    out, lse = _run(q3, p, q, d ** -0.5, 0)
    _check(p, q, out, lse, d ** -0.5, 0)

"""Residual norms on the GPU against the fp64 oracle.

Bounds: a row sum of n <= 16384 fp32 terms goes through at most 16 additions per
thread, 6 inside a wave and 16 over waves, so it is off by at most 38 * 2^-24 of
the sum of magnitudes, rounded up to 2^-18 (the reciprocal root halves that and
adds a few 2^-24).  Results add the rounding of their type: 2^-8 (bf16)."""
import numpy as np
import pytest
import torch

from oracle import q3_block as blk

pytestmark = pytest.mark.gpu

U = 2.0 ** -18
BF = 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def h64(t):
    return t.detach().double().cpu().numpy()


def make(m, n, rt, post, gate, seed=0, pitch=0):
    g = torch.Generator().manual_seed(seed)
    rows = lambda dt=torch.float32: torch.randn(m, n + pitch, generator=g).to(dt).cuda()[:, :n]  # noqa: E731
    return dict(r=rows(TYPES[rt]), pre_weight=1 + 0.3 * torch.randn(n, generator=g).cuda(), y=rows() * 2,
                post_weight=1 + 0.3 * torch.randn(n, generator=g).cuda() if post else None,
                gate={"none": None, "row": torch.randn(n, generator=g).cuda(), "full": rows()}[gate])


def ref(v):
    return {k: None if t is None else h64(t) for k, t in v.items()}


def check_forward(q3, v, scale=0.7, eps=1e-6, **kw):
    r, x = q3.q3_residual_norm(**v, scale=scale, eps=eps, **kw)
    f = ref(v)
    ro, xo = blk.residual_norm(f["r"], f["pre_weight"], f["y"], f["post_weight"], f["gate"], scale, eps)
    add = np.zeros_like(ro)
    if f["y"] is not None:   # magnitude of the block's term
        add = np.abs(ro - f["r"])
    er = 4 * 2.0 ** -24 * (np.abs(f["r"]) + add) + U * add
    root = 1 / np.sqrt((ro * ro).mean(1, keepdims=True) + eps)
    w = 1.0 if f["pre_weight"] is None else np.abs(f["pre_weight"])
    # a relative change of the row's 2-norm moves the root by as much
    row = np.sqrt((er * er).mean(1, keepdims=True)) * root
    ex = w * root * er + np.abs(xo) * (row + 2 * U + BF)
    br = BF * np.abs(ro) if v["r"].dtype == torch.bfloat16 else 0
    assert (np.abs(h64(r) - ro) <= er * (1 + BF) + br + 1e-30).all()
    assert (np.abs(h64(x) - xo) <= ex * (1 + BF) + 1e-30).all()
    return r, x


def check_backward(q3, v, dx, dr, scale=0.7, eps=1e-6, **kw):
    v = dict(v)
    kept = v.pop("r")
    g = q3.q3_residual_norm_backward(kept, dx=dx, dr_out=dr, scale=scale, eps=eps, **v, **kw)
    f = ref(v)
    out = h64(kept)
    dxh, drh = (None if t is None else h64(t) for t in (dx, dr))
    o = blk.residual_norm_backward(out, f["pre_weight"], dxh, drh, f["y"], f["post_weight"], f["gate"], scale, eps)
    bf = kept.dtype == torch.bfloat16
    n = out.shape[1]
    s = 1 / np.sqrt((out * out).mean(1, keepdims=True) + eps)
    z = np.zeros_like(out)
    a = np.abs(dxh * (1.0 if f["pre_weight"] is None else f["pre_weight"])) if dx is not None else z
    h = np.abs(out) * s
    # magnitudes of what is added up in G; its error is a few U of them
    mag = (np.abs(drh) if dr is not None else z) + s * (a + h * (a * h).sum(1, keepdims=True) / n)
    e = 4 * U * mag
    assert (np.abs(h64(g.dr) - o["dr"]) <= e + (BF * (np.abs(o["dr"]) + e) if bf else 0) + 1e-30).all()
    m = out.shape[0]
    col = 4 * U + m * 2.0 ** -24   # a column sum adds at most m terms in sequence

    def columns(name, got, terms):
        assert (np.abs(h64(got) - o[name]) <= col * terms.sum(0) + 1e-30).all(), name
    columns("dpre_weight", g.dpre_weight, (np.abs(dxh) if dx is not None else z) * h)
    if v["y"] is None:
        assert g.dy is None and g.dgate is None and g.dpost_weight is None
        return g
    up = abs(scale) * mag * (1.0 if f["gate"] is None else np.abs(f["gate"]))
    if v["post_weight"] is not None:
        sy = 1 / np.sqrt((f["y"] ** 2).mean(1, keepdims=True) + eps)
        yh = np.abs(f["y"]) * sy
        b = up * np.abs(f["post_weight"])
        size = sy * (b + yh * (b * yh).sum(1, keepdims=True) / n)
        t = yh * np.abs(f["post_weight"])
        columns("dpost_weight", g.dpost_weight, up * yh * 2)
    else:
        size, t = up, np.abs(f["y"])
    assert (np.abs(h64(g.dy) - o["dy"]) <= 8 * U * size + BF * (np.abs(o["dy"]) + 8 * U * size) + 1e-30).all()
    if v["gate"] is not None:
        terms = abs(scale) * mag * t
        if v["gate"].dim() == 1:
            columns("dgate", g.dgate, terms * 2)
        else:
            assert (np.abs(h64(g.dgate) - o["dgate"]) <= 8 * U * terms + 1e-30).all()
    return g


# every thread-group size (n up to 512, 1024, ..., 16384), columns that do and do not move in vectors
SIZES = [(1, 1), (3, 2), (5, 64), (7, 99), (9, 512), (4, 513), (3, 1024), (6, 2048), (2, 4095), (3, 4096), (2, 5120),
         (2, 8192), (3, 8191), (2, 8196), (300, 8200), (3, 12288), (2, 12287), (2, 12292), (1, 16384), (2, 16383)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_forward_sizes(q3, m, n, rt):
    check_forward(q3, make(m, n, rt, True, "full", seed=n))


@pytest.mark.parametrize("m,n", [(5, 64), (130, 260), (3, 1000)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_forms(q3, m, n, post, gate, rt):
    v = make(m, n, rt, post, gate, seed=7)
    check_forward(q3, v)
    g = torch.Generator().manual_seed(1)
    check_backward(q3, v, torch.randn(m, n, generator=g).cuda(), torch.randn(m, n, generator=g).to(TYPES[rt]).cuda())


@pytest.mark.parametrize("m,n", SIZES + [(700, 96), (5000, 64), (300, 4096)])
@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_backward_sizes(q3, m, n, rt):
    v = make(m, n, rt, True, "row", seed=n + 1)
    g = torch.Generator().manual_seed(2)
    check_backward(q3, v, torch.randn(m, n, generator=g).cuda(), torch.randn(m, n, generator=g).to(TYPES[rt]).cuda())


@pytest.mark.parametrize("rt", ["bf16", "f32"])
def test_without_block_and_partial_gradients(q3, rt):
    m, n = 6, 200
    v = make(m, n, rt, False, "none", seed=3)
    v["y"] = None
    r, x = check_forward(q3, v)
    assert r is v["r"]
    other = torch.empty_like(v["r"])
    r2, x2 = q3.q3_residual_norm(**v, scale=0.7, r_out=other)
    assert r2 is other and torch.equal(other, v["r"]) and torch.equal(x, x2)
    dx, dr = torch.randn(m, n).cuda(), torch.randn(m, n).to(TYPES[rt]).cuda()
    check_backward(q3, v, dx, None)
    check_backward(q3, v, None, dr)
    v["pre_weight"] = None
    check_forward(q3, v)
    check_backward(q3, v, dx, dr)


@pytest.mark.parametrize("pitch", [4, 5, 8])
def test_pitched_rows_and_untouched_padding(q3, pitch):
    m, n = 5, 132
    v = make(m, n, "bf16", True, "full", seed=4, pitch=pitch)
    wide_r = torch.full((m, n + pitch), 7.0, dtype=torch.bfloat16, device="cuda")
    wide_x = torch.full((m, n + pitch), 9.0, dtype=torch.bfloat16, device="cuda")
    check_forward(q3, v, r_out=wide_r[:, :n], x=wide_x[:, :n])
    assert (wide_r[:, n:] == 7).all() and (wide_x[:, n:] == 9).all()
    g = check_backward(q3, v, torch.randn(m, n + pitch).cuda()[:, :n], None)
    # vectors and single elements give the same sums only to rounding, the same call the same bits
    g2 = check_backward(q3, v, torch.zeros(m, n).cuda(), torch.randn(m, n).to(torch.bfloat16).cuda())
    assert g.dr.shape == g2.dr.shape


def test_in_place_residual(q3):
    v = make(9, 300, "bf16", True, "row", seed=5)
    r, x = q3.q3_residual_norm(**v, scale=0.5)
    r2, x2 = q3.q3_residual_norm(**v, scale=0.5, r_out=v["r"])
    assert r2 is v["r"] and torch.equal(r, r2) and torch.equal(x, x2)


def test_zero_rows_and_repeated_calls(q3):
    v = make(64, 1024, "f32", True, "row", seed=6)
    v["y"][3] = 0
    v["r"][3] = 0
    check_forward(q3, v)
    dx = torch.randn(64, 1024).cuda()
    a = check_backward(q3, v, dx, dx)
    b = check_backward(q3, v, dx, dx)
    for k in ("dr", "dy", "dgate", "dpost_weight", "dpre_weight"):
        assert torch.equal(getattr(a, k), getattr(b, k)), k


def test_rows_do_not_meet(q3):
    # a row of NaN stays alone, whatever its neighbours share with it
    for n in (64, 512, 2000):
        v = make(9, n, "f32", True, "full", seed=8)
        base = [t.clone() for t in q3.q3_residual_norm(**v)]
        v["y"][4, 1] = float("nan")
        r, x = q3.q3_residual_norm(**v)
        keep = [i for i in range(9) if i != 4]
        assert torch.equal(r[keep], base[0][keep]) and torch.equal(x[keep], base[1][keep])
        assert torch.isnan(x[4]).all()


def test_binding_refusals(q3):
    r = torch.zeros(2, 64, device="cuda")
    with pytest.raises(ValueError):
        q3.q3_residual_norm(r, gate=torch.zeros(64, device="cuda"))            # a gate without y
    with pytest.raises(ValueError):
        q3.q3_residual_norm(r, y=torch.zeros(2, 63, device="cuda"))
    with pytest.raises(ValueError):
        q3.q3_residual_norm(r, pre_weight=torch.zeros(64))                     # on the host
    with pytest.raises(ValueError):
        q3.q3_residual_norm(r.half())
    with pytest.raises(q3.Q3Error):
        q3.q3_residual_norm(torch.zeros(1, 16385, device="cuda"))

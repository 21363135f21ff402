"""Products of many tokens and the gated feed-forward block on the GPU against
the fp64 oracle.

Bounds: products of bf16 values are exact in fp32; k of them are added with at
most k roundings of 2^-23 (the matrix cores may truncate), so |y - ref| <=
k 2^-23 sum|x w|.  Activations are good to 16 * 2^-24 and their slope stays below
1.13 in magnitude; results in bf16 add half a step, 2^-8."""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import pack_layer
from oracle import q3_block as blk

pytestmark = pytest.mark.gpu
BF = 2.0 ** -8


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def h64(t):
    return t.detach().double().cpu().numpy()


def weights(layer):
    return oracle.dequantize(layer.codes, layer.scales, layer.codebook)


def tokens(m, cols, seed, pitch=0):
    g = torch.Generator().manual_seed(seed)
    wide = (cols + 7) // 8 * 8 + 8 * pitch
    t = torch.full((m, wide), float("nan"), dtype=torch.bfloat16)   # what stands behind the rows is not read
    t[:, :cols] = torch.randn(m, cols, generator=g).to(torch.bfloat16)
    return t.cuda()[:, :cols]


def check_product(got, a, w, extra=None):
    """got = a w^T within k 2^-23 sum|a||w|."""
    ref, mag = a @ w.T, np.abs(a) @ np.abs(w.T)
    assert got.shape == ref.shape
    assert (np.abs(h64(got) - ref) <= a.shape[1] * 2.0 ** -23 * mag + 1e-30).all()


# rows that end inside tiles of 16, 64, 128 and 256, k that ends inside a 64- and a 512-step
SHAPES = [(1, 32, 1), (5, 96, 3), (16, 64, 65), (45, 160, 100), (64, 512, 70), (100, 544, 129), (130, 1024, 200),
          (256, 2080, 64), (257, 320, 257), (300, 4096, 66), (1000, 96, 500), (512, 512, 1),
          # few tiles and a long summed axis: split (forwards, backwards, both), ragged columns
          (130, 4128, 100), (4100, 96, 100), (2045, 2080, 130)]


@pytest.mark.parametrize("n,k,m", SHAPES)
def test_gemm_both_ways(q3, n, k, m):
    layer = synth.make_layer(n, k, seed=n + k)
    w, w64 = pack_layer(q3, layer), weights(layer)
    x, dy = tokens(m, k, 1), tokens(m, n, 2)
    check_product(q3.q3_gemm(w, x), h64(x), w64)
    check_product(q3.q3_gemm_backward(w, dy), h64(dy), w64.T)


@pytest.mark.parametrize("m", [1, 16, 17, 63, 64, 65, 127, 128, 255, 256, 511, 1025])
def test_gemm_token_counts(q3, m):
    n, k = 320, 672
    layer = synth.make_layer(n, k, seed=5)
    w, w64 = pack_layer(q3, layer), weights(layer)
    x, dy = tokens(m, k, 3), tokens(m, n, 4)
    check_product(q3.q3_gemm(w, x), h64(x), w64)
    check_product(q3.q3_gemm_backward(w, dy), h64(dy), w64.T)


@pytest.mark.parametrize("n,k,m", [(1024, 8192, 1600), (8200, 1024, 1500)])
def test_gemm_large_tiles(q3, n, k, m):
    # enough tiles for the large-block kernel; a sample of rows against the oracle
    layer = synth.make_layer(n, k, seed=9)
    w, w64 = pack_layer(q3, layer), weights(layer)
    x, dy = tokens(m, k, 5), tokens(m, n, 6)
    rows = [0, 1, 255, 256, 700, m - 1]
    check_product(q3.q3_gemm(w, x)[rows], h64(x[rows]), w64)
    check_product(q3.q3_gemm_backward(w, dy)[rows], h64(dy[rows]), w64.T)


@pytest.mark.parametrize("n,m", [(9232, 70), (9232, 128), (9232, 129), (18500, 250), (40000, 513), (9408, 70),
                                 (9408, 128), (9408, 129), (18816, 250), (40000, 445)])
def test_gemm_tall_matrix_in_passes(q3, n, m):
    # tall matrices take 64 tokens at a time from the packed planes, up to a number that grows with n
    k = 96
    layer = synth.make_layer(n, k, seed=3)
    w, w64 = pack_layer(q3, layer), weights(layer)
    x = tokens(m, k, 1, pitch=1)
    check_product(q3.q3_gemm(w, x), h64(x), w64)


@pytest.mark.parametrize("n,k", [(16, 512), (45, 1024), (300, 1536), (1000, 4096), (4100, 2560), (9000, 512)])
def test_gemm_of_65_to_128_tokens(q3, n, k):
    # whole steps of K, split over blocks (evenly or not) or not; the last pass of more tokens
    layer = synth.make_layer(n, k, seed=n)
    w, w64 = pack_layer(q3, layer), weights(layer)
    for m in (65, 80, 96, 97, 112, 127, 128, 129, 200):
        x = tokens(m, k, m, pitch=1)
        y = torch.full((m, n + 3), 5.0, device="cuda")
        check_product(q3.q3_gemm(w, x, y=y[:, :n]), h64(x), w64)
        assert (y[:, n:] == 5).all()
        need = q3.q3_gemm_workspace_bytes(n, k, m)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(q3.q3_gemm(w, x, workspace=ws[:need]), q3.q3_gemm(w, x)) and (ws[need:] == 255).all()
        bad = x.clone()
        bad[3] = float("nan")
        got, rows = q3.q3_gemm(w, bad), [i for i in range(m) if i != 3]
        assert torch.equal(got[rows], q3.q3_gemm(w, x)[rows]) and got[3].isnan().all()


@pytest.mark.parametrize("inter,k", [(32, 512), (96, 1024), (160, 2560), (10016, 512)])
def test_glu_of_65_to_128_tokens(q3, inter, k):
    w, w64 = glu_case(q3, inter, k, seed=inter)
    for m in (65, 96, 97, 128, 129, 260):
        h = torch.full((m, inter + 8), 5.0, dtype=torch.bfloat16, device="cuda")
        check_glu(q3, w, w64, tokens(m, k, m, pitch=1), "gelu", h=h[:, :inter])
        assert (h[:, inter:] == 5).all()


@pytest.mark.parametrize("inter,m", [(4640, 70), (4640, 128), (4640, 129), (9248, 250), (4704, 70), (4704, 128),
                                     (4704, 129), (9408, 250)])
def test_glu_tall_matrix_in_passes(q3, inter, m):
    w, w64 = glu_case(q3, inter, 96, seed=3)
    check_glu(q3, w, w64, tokens(m, 96, 1), "silu")


def test_gemm_pitched_rows(q3):
    n, k, m = 77, 160, 90
    layer = synth.make_layer(n, k, seed=2)
    w, w64 = pack_layer(q3, layer), weights(layer)
    x, dy = tokens(m, k, 7, pitch=3), tokens(m, n, 8, pitch=2)
    for pitch in (3, 4):
        y = torch.full((m, n + pitch), 5.0, device="cuda")
        dx = torch.full((m, k + pitch), 6.0, device="cuda")
        check_product(q3.q3_gemm(w, x, y=y[:, :n]), h64(x), w64)
        check_product(q3.q3_gemm_backward(w, dy, dx=dx[:, :k]), h64(dy), w64.T)
        assert (y[:, n:] == 5).all() and (dx[:, k:] == 6).all()


def one_infinity(rows, cols, at, seed):
    """Row i holds an infinity at column at[i % len(at)] and numbers elsewhere."""
    t = tokens(rows, cols, seed)
    for i in range(rows):
        t[i, at[i % len(at)]] = float("inf") if i % 3 else -float("inf")
    return t


@pytest.mark.parametrize("m", [3, 70, 300])
@pytest.mark.parametrize("n,k", [(45, 96), (100, 544), (200, 32)])
def test_gemm_infinities(q3, n, k, m):
    # an infinity leaves its sign (0 times it: NaN) and nothing else; columns behind a tile's end add nothing
    layer = synth.make_layer(n, k, seed=n)
    w, w64 = pack_layer(q3, layer), weights(layer)
    for cols, f, mat in ((k, q3.q3_gemm, w64), (n, q3.q3_gemm_backward, w64.T)):
        last = (cols - 1) // 64 * 64
        at = [last, min(last + 7, cols - 1), cols - 1, 0, cols // 2]
        x = one_infinity(m, cols, at, 5)
        got = h64(f(w, x))
        for i in range(m):
            a = at[i % len(at)]
            with np.errstate(invalid="ignore"):
                want = h64(x)[i, a] * mat[:, a]
            np.testing.assert_array_equal(got[i], want)


@pytest.mark.parametrize("n,k", [(64, 96), (128, 544), (128, 1120), (20032, 96), (64, 512)])
def test_one_token_not_a_number(q3, n, k):
    # the other tokens' results are what they are without it, where K ends inside a step too
    layer = synth.make_layer(n, k, seed=1)
    w = pack_layer(q3, layer)
    for m in (2, 3, 8, 9, 16, 17, 33, 49, 64, 70, 129):
        x = tokens(m, k, 1, pitch=2)   # what stands behind the rows is NaN as well
        calls = [lambda a: q3.q3_gemm(w, a), lambda a: q3.q3_glu(w, a)]
        if m <= 8:
            calls.append(lambda a: q3.q3_gemv(w, a))
        for f in calls:
            clean = f(x)
            assert torch.isfinite(clean).all()
            for bad in (0, m // 2, m - 1):
                for value in (float("nan"), float("inf")):
                    other = x.clone()
                    other[bad] = value
                    wide = torch.full((m, x.stride(0)), value, dtype=torch.bfloat16, device="cuda")
                    wide[:, :k] = other
                    for a in (other, wide[:, :k]):
                        got = f(a)
                        rows = [i for i in range(m) if i != bad]
                        assert torch.equal(got[rows], clean[rows])
                        if value != value:
                            assert got[bad].isnan().all()


def test_gemm_after_not_a_number(q3):
    # what an earlier call left in the chip's memories does not reach columns that a tile pads
    big = synth.make_layer(256, 512, seed=1)
    wb = pack_layer(q3, big)
    for m in (3, 70, 600):
        for n, k in ((45, 32), (100, 96), (300, 160)):
            layer = synth.make_layer(n, k, seed=2)
            w, w64 = pack_layer(q3, layer), weights(layer)
            x, dy = tokens(m, k, 1), tokens(m, n, 2)
            nan = torch.full((600, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
            q3.q3_gemm(wb, nan)
            check_product(q3.q3_gemm(w, x), h64(x), w64)
            q3.q3_gemm(wb, nan)
            check_product(q3.q3_gemm_backward(w, dy), h64(dy), w64.T)


def test_gemm_empty_matrix(q3):
    w = q3.empty_packed(0, 64, "cuda")
    assert q3.q3_gemm(w, tokens(70, 64, 1)).shape == (70, 0)
    dx = torch.full((70, 64), 3.0, device="cuda")
    q3.q3_gemm_backward(w, torch.empty(70, 0, dtype=torch.bfloat16, device="cuda"), dx=dx)
    assert (dx == 0).all()


def glu_case(q3, inter, k, seed=0):
    layer = synth.make_layer(2 * inter, k, seed=seed)
    return pack_layer(q3, layer), weights(layer)


def check_glu(q3, w, w64, x, act, **kw):
    inter, k = w64.shape[0] // 2, w64.shape[1]
    h, pre = q3.q3_glu(w, x, act=act, save_pre=True, **kw)
    ref, pre64 = blk.glu(w64, h64(x), act)
    e = k * 2.0 ** -23 * (np.abs(h64(x)) @ np.abs(w64.T))
    assert (np.abs(h64(pre) - pre64) <= e + 1e-30).all()
    g, u = pre64[:, :inter], pre64[:, inter:]
    eg, eu = e[:, :inter], e[:, inter:]
    a = np.abs(blk.act(act, g))
    eh = (1.13 * eg) * (np.abs(u) + eu) + a * eu + 2.0 ** -20 * a * np.abs(u)
    assert (np.abs(h64(h) - ref) <= eh + BF * (np.abs(ref) + eh) + 1e-30).all()
    assert torch.equal(h, q3.q3_glu(w, x, act=act))   # with and without the pre-activations
    return h, pre


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("inter,k", [(32, 32), (96, 160), (64, 512), (224, 2048), (160, 4096), (352, 1056)])
def test_glu_shapes(q3, inter, k, act):
    w, w64 = glu_case(q3, inter, k, seed=inter)
    for m in (1, 2, 5, 16, 17, 33, 48, 49, 64, 65, 130, 300):
        check_glu(q3, w, w64, tokens(m, k, m), act)


def test_glu_large_tiles(q3):
    inter, k, m = 2080, 512, 3000
    w, w64 = glu_case(q3, inter, k, seed=1)
    check_glu(q3, w, w64, tokens(m, k, 1), "silu")


def test_glu_wide_rows_of_activations(q3):
    # more activations than a block can hold: the streamed forms
    inter, k = 64, 8192
    w, w64 = glu_case(q3, inter, k, seed=4)
    for m in (12, 20, 40, 64):
        check_glu(q3, w, w64, tokens(m, k, m), "silu")
    w, w64 = glu_case(q3, inter, 8192 + 96, seed=4)
    for m in (12, 20, 40, 64):
        check_glu(q3, w, w64, tokens(m, 8192 + 96, m), "gelu")


def test_glu_pitched_rows(q3):
    inter, k = 96, 160
    w, w64 = glu_case(q3, inter, k, seed=2)
    for m in (3, 70):
        h = torch.full((m, inter + 8), 5.0, dtype=torch.bfloat16, device="cuda")
        pre = torch.full((m, 2 * inter + 4), 6.0, device="cuda")
        check_glu(q3, w, w64, tokens(m, k, 3, pitch=1), "silu", h=h[:, :inter], pre=pre[:, :2 * inter])
        assert (h[:, inter:] == 5).all() and (pre[:, 2 * inter:] == 6).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_backward(q3, act):
    for m, inter in ((1, 32), (3, 96), (70, 1056)):
        g = torch.Generator().manual_seed(m)
        pre = (torch.randn(m, 2 * inter, generator=g) * 4).cuda()
        dh = torch.randn(m, inter, generator=g).cuda()
        pre[0, :8] = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e5, -1e5, 3e38, -3e38])
        got, ref = h64(q3.q3_glu_backward(pre, dh, act=act)), None
        with np.errstate(all="ignore"):
            ref = blk.glu_backward(h64(pre), h64(dh), act)
        u = np.abs(h64(pre)[:, inter:])
        d = np.abs(h64(dh))
        # the slope is a difference of terms up to |z| <= ~10 in size where it is not 0 or 1
        bound = np.concatenate([d * u * 64 * 2.0 ** -23, 2.0 ** -20 * np.abs(ref[:, inter:])], 1) + BF * np.abs(ref)
        fin = np.isfinite(ref) & (np.abs(ref) < 3.3e38)
        assert (np.abs(got - ref)[fin] <= bound[fin] + 1e-30).all()
        assert not np.isnan(got).any()


def test_whole_block_against_differences(q3):
    # h and its gradient in x through the packed weights, as a training step chains them
    inter, k, m = 64, 96, 70
    gu, gu64 = glu_case(q3, inter, k, seed=3)
    layer = synth.make_layer(k, inter, seed=4)
    dn, dn64 = pack_layer(q3, layer), weights(layer)
    x, dy = tokens(m, k, 1), tokens(m, k, 2)
    h, pre = q3.q3_glu(gu, x, save_pre=True)
    y = q3.q3_gemm(dn, h)
    dh = q3.q3_gemm_backward(dn, dy)
    dpre = q3.q3_glu_backward(pre, dh)
    dx = h64(q3.q3_gemm_backward(gu, dpre))
    x64, dy64 = h64(x), h64(dy)
    f = lambda v: (blk.glu(gu64, v, "silu")[0] @ dn64.T * dy64).sum(1)  # noqa: E731  (per token)
    # dpre is rounded to bf16: |error| <= 2^-8 |dpre| |w| and the products' own
    size = np.abs(blk.glu_backward(blk.glu(gu64, x64, "silu")[1], dy64 @ dn64, "silu")) @ np.abs(gu64)
    for j in range(0, k, 7):
        d = np.zeros_like(x64)
        d[:, j] = 1e-4
        num = (f(x64 + d) - f(x64 - d)) / 2e-4
        assert (np.abs(dx[:, j] - num) <= (BF + 1e-4) * size[:, j] + 1e-4 * (1 + np.abs(num))).all()
    assert y.shape == (m, k)


def test_captured_and_replayed(q3):
    # both lengths' kernels under one graph, with eager work between the replays
    inter, k = 96, 160
    w, _ = glu_case(q3, inter, k, seed=6)
    layer = synth.make_layer(k, inter, seed=7)
    dn = pack_layer(q3, layer)
    for m in (4, 200):
        x, dh = tokens(m, k, 1).contiguous(), torch.randn(m, inter, device="cuda")

        def step():
            h, pre = q3.q3_glu(w, x, save_pre=True)
            y = q3.q3_gemm(dn, h)
            dpre = q3.q3_glu_backward(pre, dh)
            return h, pre, y, dpre, q3.q3_gemm_backward(w, dpre)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        for i in range(3):
            x.copy_(torch.randn(m, k, device="cuda"))
            dh.copy_(torch.randn(m, inter, device="cuda"))
            g.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            for a, b in zip(got, step()):
                assert torch.equal(a, b)
            torch.zeros(1000, device="cuda").sum().item()


def test_workspaces(q3):
    n, k, m = 128, 160, 100
    layer = synth.make_layer(n, k, seed=8)
    w = pack_layer(q3, layer)
    x, dy = tokens(m, k, 1), tokens(m, n, 2)
    for f, size, a in ((q3.q3_gemm, q3.q3_gemm_workspace_bytes, x),
                       (q3.q3_gemm_backward, q3.q3_gemm_backward_workspace_bytes, dy),
                       (q3.q3_glu, q3.q3_glu_workspace_bytes, x)):
        nbytes = size(n, k, m)
        ws = torch.full((nbytes + 512,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(f(w, a, workspace=ws[:nbytes]), f(w, a))
        assert (ws[nbytes:] == 255).all()                                    # nothing past the stated size
        with pytest.raises(q3.Q3Error):
            f(w, a, workspace=ws[:nbytes - 256])
        with pytest.raises(q3.Q3Error):
            f(w, a, workspace=ws[64:nbytes + 64])


def test_binding_refusals(q3):
    layer = synth.make_layer(128, 64, seed=8)
    w = pack_layer(q3, layer)
    x = tokens(4, 64, 1)
    with pytest.raises(ValueError):
        q3.q3_gemm(w, x.float())
    with pytest.raises(ValueError):
        q3.q3_gemm(w, x[:, :32])
    with pytest.raises(ValueError):
        q3.q3_gemm(w, x, y=torch.empty(3, 128, device="cuda"))
    with pytest.raises(ValueError):
        q3.q3_glu(w, x, act="tanh")
    with pytest.raises(ValueError):
        q3.q3_glu_backward(torch.zeros(2, 128, device="cuda"), torch.zeros(2, 32, device="cuda"))
    with pytest.raises(q3.Q3Error):
        q3.q3_gemm(w, x[:0])
    with pytest.raises(q3.Q3Error):
        q3.q3_glu_backward(torch.zeros(2, 96, device="cuda"), torch.zeros(2, 48, device="cuda"))
    odd = synth.make_layer(96, 64, seed=8)                                     # I = 48
    with pytest.raises(q3.Q3Error):
        q3.q3_glu(pack_layer(q3, odd), x)

"""The operators of include/q3_block.h run together, as a decode step and a
training step use them, on the GPU: the feed-forward sublayer against its parts
and the fp64 oracle, a step from residual stream to token, a training step
against differences, captured graphs, streams and tensors past 32 bits.

Bounds: a product's as in test_gpu_ffn.py, k 2^-23 sum|x w|; half a step of bf16,
2^-8, for every bf16 result on the way."""
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


def gen(*shape, seed, scale=1.0, base=0.0):
    g = torch.Generator().manual_seed(seed)
    return (base + scale * torch.randn(*shape, generator=g)).cuda()


class Block:
    """Packed gate_up [2I][k] and down [k][I], and the norm weights."""

    def __init__(self, q3, k, inter, seed=0):
        gu, dn = synth.make_layer(2 * inter, k, seed=seed), synth.make_layer(k, inter, seed=seed + 1)
        self.gu, self.dn = pack_layer(q3, gu), pack_layer(q3, dn)
        self.gu64 = oracle.dequantize(gu.codes, gu.scales, gu.codebook)
        self.dn64 = oracle.dequantize(dn.codes, dn.scales, dn.codebook)
        self.pre, self.post, self.next = (gen(k, seed=seed + i, scale=0.2, base=1.0) for i in (2, 3, 4))
        self.k, self.inter = k, inter


def parts(q3, b, r, gate, scale, act, eps=1e-6, post=True, nxt=True):
    """The sublayer by its separate calls."""
    _, x = q3.q3_residual_norm(r, b.pre, eps=eps)
    h = q3.q3_glu(b.gu, x, act=act)
    y = q3.q3_gemm(b.dn, h)
    return q3.q3_residual_norm(r, b.next if nxt else None, y, b.post if post else None, gate, scale, eps)


CASES = [(64, 32, 1), (96, 160, 3), (96, 160, 64), (96, 160, 65), (512, 1056, 17), (2080, 64, 200), (160, 4640, 100),
         (4096, 4096, 1)]


@pytest.mark.parametrize("k,inter,m", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ffn_is_its_parts(q3, k, inter, m, dtype):
    b = Block(q3, k, inter)
    r = gen(m, k, seed=9).to(dtype)
    for gate, scale, act, post, nxt in ((None, 1.0, "silu", True, True), (gen(k, seed=8), 0.5, "gelu", False, True),
                                        (gen(m, k, seed=8), 2.0, "silu", True, False)):
        kw = dict(post_weight=b.post if post else None, gate=gate, scale=scale, act=act,
                  next_weight=b.next if nxt else None)
        want = parts(q3, b, r, gate, scale, act, post=post, nxt=nxt)
        for got in (q3.q3_ffn(b.gu, b.dn, r, b.pre, **kw), q3.q3_ffn(b.gu, b.dn, r.clone(), b.pre, **kw)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        own = r.clone()                                                     # r_out in place
        got = q3.q3_ffn(b.gu, b.dn, own, b.pre, r_out=own, **kw)
        assert got[0] is own and torch.equal(own, want[0]) and torch.equal(got[1], want[1])


def test_ffn_against_the_oracle(q3):
    # eps large enough that no norm amplifies: each rounding is then carried on by at most its own size
    k, inter, m = 160, 96, 70
    b = Block(q3, k, inter, seed=3)
    r = gen(m, k, seed=1)
    r64 = h64(r)
    got = h64(q3.q3_ffn(b.gu, b.dn, r, b.pre, None, None, 1.0, b.next)[0])
    _, x = blk.residual_norm(r64, h64(b.pre))
    h, pre = blk.glu(b.gu64, x, "silu")
    y = h @ b.dn64.T
    # x is off by (2^-8 + 2^-20)|x|, so pre by e; h by its slope (below 1.13) and its own rounding; y by their sums
    e = (BF + 2.0 ** -18) * (np.abs(x) @ np.abs(b.gu64.T))
    g, u, eg, eu = pre[:, :inter], pre[:, inter:], e[:, :inter], e[:, inter:]
    eh = 1.13 * eg * (np.abs(u) + eu) + np.abs(blk.act("silu", g)) * eu
    eh = eh + (BF + 2.0 ** -18) * (np.abs(h) + eh)
    ey = (eh + 2.0 ** -16 * np.abs(h)) @ np.abs(b.dn64.T)
    assert (np.abs(got - (r64 + y)) <= ey + 2.0 ** -23 * np.abs(r64 + y)).all()


def test_ffn_rows_apart_and_pitched(q3):
    k, inter = 96, 64
    b = Block(q3, k, inter, seed=5)
    for m in (5, 90):
        wide = gen(m, k + 8, seed=2)
        want = q3.q3_ffn(b.gu, b.dn, wide[:, :k].contiguous(), b.pre, b.post, None, 1.0, b.next)
        r_out = torch.full((m, k + 4), 7.0, device="cuda")
        x = torch.full((m, k + 8), 5.0, dtype=torch.bfloat16, device="cuda")
        q3.q3_ffn(b.gu, b.dn, wide[:, :k], b.pre, b.post, None, 1.0, b.next, r_out=r_out[:, :k], x=x[:, :k])
        assert torch.equal(r_out[:, :k], want[0]) and torch.equal(x[:, :k], want[1])
        assert (r_out[:, k:] == 7).all() and (x[:, k:] == 5).all()
        bad = wide[:, :k].contiguous()
        bad[2] = float("nan")                                                # one token's NaN stays its own
        got = q3.q3_ffn(b.gu, b.dn, bad, b.pre, b.post, None, 1.0, b.next)
        rows = [i for i in range(m) if i != 2]
        assert torch.equal(got[0][rows], want[0][rows]) and got[0][2].isnan().all() and got[1][2].isnan().all()


def test_ffn_workspace_and_refusals(q3):
    b = Block(q3, 96, 64, seed=5)
    for m in (3, 100):
        r = gen(m, 96, seed=2)
        need = q3.q3_ffn_workspace_bytes(128, 96, m)
        ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
        want = q3.q3_ffn(b.gu, b.dn, r, b.pre)
        got = q3.q3_ffn(b.gu, b.dn, r, b.pre, workspace=ws[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (ws[need:] == 255).all()
        with pytest.raises(q3.Q3Error):
            q3.q3_ffn(b.gu, b.dn, r, b.pre, workspace=ws[:need - 256])
    r = gen(3, 96, seed=2)
    for bad in (lambda: q3.q3_ffn(b.gu, b.gu, r), lambda: q3.q3_ffn(b.gu, b.dn, r[:, :64]),
                lambda: q3.q3_ffn(b.gu, b.dn, r.half()), lambda: q3.q3_ffn(b.gu, b.dn, r, b.pre[:64]),
                lambda: q3.q3_ffn(b.gu, b.dn, r, gate=gen(2, 96, seed=1)),
                lambda: q3.q3_ffn(b.gu, b.dn, r, next_weight=b.next.double()),
                lambda: q3.q3_ffn(b.gu, b.dn, r, act="relu"), lambda: q3.q3_ffn(b.gu, b.dn, r.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q3.Q3Error):
        q3.q3_ffn(b.gu, b.dn, r[:0])


def decode(q3, blocks, head, r, u, final):
    """Residual stream -> token: every block, the last norm, the vocabulary product, the choice."""
    for b in blocks:
        r, x = q3.q3_ffn(b.gu, b.dn, r, b.pre, b.post, None, 1.0, final)
    logits = q3.q3_gemm(head, x)
    return (r, x, logits) + q3.q3_sample(logits, u, top_p=torch.full_like(u, 0.9), temperature=torch.full_like(u, 0.7))


@pytest.mark.parametrize("m", [1, 5, 64, 70])
def test_decode_step(q3, m):
    k, n = 160, 1000
    blocks = [Block(q3, k, 96, seed=s) for s in (0, 10)]
    layer = synth.make_layer(n, k, seed=20)
    head, head64 = pack_layer(q3, layer), oracle.dequantize(layer.codes, layer.scales, layer.codebook)
    r, u = gen(m, k, seed=30).to(torch.bfloat16), torch.rand(m, generator=torch.Generator().manual_seed(1)).cuda()
    final = gen(k, seed=31, scale=0.1, base=1.0)
    r2, x, logits, tok, lp = decode(q3, blocks, head, r, u, final)
    ref, mag = h64(x) @ head64.T, np.abs(h64(x)) @ np.abs(head64.T)
    assert (np.abs(h64(logits) - ref) <= k * 2.0 ** -23 * mag).all()
    for i in range(m):
        t, p = blk.sample(h64(logits)[i], float(u[i]), float(np.float32(0.7)), 0, float(np.float32(0.9)))
        # fp32 rounding of the result and 2^-45 for each of n weights against a sum of at least 1
        assert int(tok[i]) == t and abs(float(lp[i]) - p) <= 2.0 ** -23 * abs(p) + 2e-7


def test_decode_step_captured(q3):
    k, n, m = 96, 500, 4
    blocks = [Block(q3, k, 64, seed=s) for s in (0, 10)]
    head = pack_layer(q3, synth.make_layer(n, k, seed=20))
    r, u = gen(m, k, seed=30), torch.rand(m, device="cuda")
    final = torch.ones(k, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        decode(q3, blocks, head, r, u, final)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = decode(q3, blocks, head, r, u, final)
    for i in range(4):
        r.copy_(gen(m, k, seed=50 + i))
        u.copy_(torch.rand(m, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, decode(q3, blocks, head, r, u, final)):
            assert torch.equal(a, b)
        torch.zeros(1000, device="cuda").sum().item()


def train(q3, b, r, dr_out, dx_next, gate):
    """One sublayer forward and backward -> (r', x', gradients of r, the weights and the gate)."""
    _, x = q3.q3_residual_norm(r, b.pre)
    h, pre = q3.q3_glu(b.gu, x, save_pre=True)
    y = q3.q3_gemm(b.dn, h)
    r1, x1 = q3.q3_residual_norm(r, b.next, y, b.post, gate, 0.5)
    back = q3.q3_residual_norm_backward(r1, b.next, dx_next, dr_out, y, b.post, gate, 0.5)
    dh = q3.q3_gemm_backward(b.dn, back.dy)
    dpre = q3.q3_glu_backward(pre, dh)
    dx = q3.q3_gemm_backward(b.gu, dpre)
    first = q3.q3_residual_norm_backward(r, b.pre, dx, back.dr)
    return r1, x1, first.dr, first.dpre_weight, back.dpre_weight, back.dpost_weight, back.dgate


def plain_norm(v, w, eps=1e-6):
    n = v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    return n * w, n


def plain_norm_back(v, w, dx, eps=1e-6):
    s = torch.rsqrt((v * v).mean(1, keepdim=True) + eps)
    a, n = dx * w, v * s
    return s * (a - n * (a * n).mean(1, keepdim=True)), (dx * n).sum(0)


def plain_train(b, r, dr_out, dxn, gate, pre_w, post_w, nxt_w, off):
    """train() in fp64 by the formulas, with the four roundings to bf16 as relative offsets."""
    gu, dn = torch.tensor(b.gu64), torch.tensor(b.dn64)
    x = plain_norm(r, pre_w)[0] * (1 + off[0])
    g, u = (x @ gu.T).chunk(2, 1)
    sig = torch.sigmoid(g)
    y = (g * sig * u * (1 + off[1])) @ dn.T
    t, _ = plain_norm(y, post_w)
    r1 = r + 0.5 * gate * t
    back, dnext = plain_norm_back(r1, nxt_w, dxn)
    dr1 = dr_out + back
    dgate = (0.5 * dr1 * t).sum(0)
    dy, dpost = plain_norm_back(y, post_w, 0.5 * dr1 * gate)
    dh = (dy * (1 + off[2])) @ dn
    dpre = torch.cat([dh * u * (sig + g * sig * (1 - sig)), dh * g * sig], 1) * (1 + off[3])
    first, dpre_w = plain_norm_back(r, pre_w, dpre @ gu)
    loss = (r1 * dr_out).sum() + (plain_norm(r1, nxt_w)[0] * dxn).sum()
    return loss, {"r": dr1 + first, "pre": dpre_w, "nxt": dnext, "post": dpost, "gate": dgate}


@pytest.mark.parametrize("m", [3, 70])
def test_training_step_against_formula_and_differences(q3, m):
    k, inter = 96, 64
    b = Block(q3, k, inter, seed=7)
    r, dr_out, dxn, gate = gen(m, k, seed=1), gen(m, k, seed=2), gen(m, k, seed=3), gen(k, seed=4)
    _, _, *got = train(q3, b, r, dr_out, dxn, gate)
    got = dict(zip(("r", "pre", "nxt", "post", "gate"), got))
    c = lambda t: t.double().cpu()  # noqa: E731
    at = {"r": c(r), "pre": c(b.pre), "nxt": c(b.next), "post": c(b.post), "gate": c(gate)}
    off = [torch.zeros(m, n, dtype=torch.float64, requires_grad=True) for n in (k, inter, k, 2 * inter)]
    run = lambda v, o: plain_train(b, v["r"], c(dr_out), c(dxn), v["gate"], v["pre"], v["post"], v["nxt"], o)  # noqa: E731
    _, grads = run(at, off)
    for name, want in grads.items():
        for seed in range(3):
            d = torch.randn(want.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
            along = (want * d).sum()
            e = 1e-6
            up, down = (run(dict(at, **{name: at[name] + s * d}), [0.0] * 4)[0] for s in (e, -e))
            assert abs(along.item() - ((up - down) / (2 * e)).item()) <= 1e-5 * (1 + abs(along.item()))
            # first order: 2^-8 for each rounding; a tenth more for the second order and fp32
            carried = sum(t.abs().sum().item() for t in torch.autograd.grad(along, off, retain_graph=True,
                                                                            allow_unused=True) if t is not None)
            fp32 = 2.0 ** -16 * (want.abs() * d.abs()).sum().item()
            assert abs((c(got[name]) * d).sum().item() - along.item()) <= 1.1 * BF * carried + fp32, (name, seed)


def test_training_step_captured_beside_an_eager_one(q3):
    # two graphs with their own memory, replayed on two streams at once, and the eager step between
    k, inter, m = 96, 64, 70
    b = Block(q3, k, inter, seed=7)
    ins = [[gen(m, k, seed=10 * j + i) for i in range(3)] + [gen(k, seed=10 * j + 3)] for j in range(2)]
    eager = train(q3, b, *ins[0])
    graphs, outs = [], []
    for j in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(train(q3, b, *ins[j]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(3):
        for j in range(2):
            ins[j][0].copy_(gen(m, k, seed=90 + 2 * i + j))
        torch.cuda.synchronize()
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                graphs[j].replay()
        torch.cuda.synchronize()
        for j in range(2):
            for a, e in zip(outs[j], train(q3, b, *ins[j])):
                assert torch.equal(a, e)
    assert all(torch.isfinite(t).all() for t in eager)


def test_calls_on_another_stream(q3):
    # inputs made on one stream, the call on another that waits for it
    k, m = 4096, 512
    w = gen(k, seed=1)
    s = torch.cuda.Stream()
    for i in range(3):
        r = gen(m, k, seed=2 + i)
        y = gen(m, k, seed=20 + i)
        torch.cuda.synchronize()
        want = q3.q3_residual_norm(r, w, y)
        r2, y2 = r * 1.0, y * 1.0
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got = q3.q3_residual_norm(r2, w, y2)
            back = q3.q3_residual_norm_backward(got[0], w, y2, None, y2)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        again = q3.q3_residual_norm_backward(want[0], w, y, None, y)
        assert torch.equal(back.dr, again.dr) and torch.equal(back.dpre_weight, again.dpre_weight)


def random_planes(q3, n, k, seed):
    """A packed matrix of random codes and moderate scales, made on the device."""
    w = q3.empty_packed(n, k, "cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    w.code_plane.random_(0, 256, generator=g)
    w.scale_plane.random_(118, 123, generator=g)
    w.codebook.random_(0x28, 0x48, generator=g)                       # finite E4M3, 0.25 .. 3.75
    w.codebook |= (torch.randint(0, 2, w.codebook.shape, generator=g, device="cuda", dtype=torch.uint8) << 7)
    return w


def last_rows(q3, w, rows):
    """The matrix of the last `rows` rows (planes lie row tile by row tile)."""
    tiles = rows // 16
    t = w.n // 16
    part = q3.empty_packed(rows, w.k, "cuda")
    for name in ("code_plane", "scale_plane"):
        whole, small = getattr(w, name).view(-1), getattr(part, name).view(-1)
        small.copy_(whole[whole.numel() // t * (t - tiles):])
    part.codebook.copy_(w.codebook[-rows:])
    return part


def test_offsets_past_32_bits(q3):
    # widened weights of 4.9 GB, outputs of 9.7 GB: the last rows against the product of those rows alone
    n, k, m, rows = 302_000 // 64 * 64, 8192, 8000, 64
    w = random_planes(q3, n, k, 1)
    part = last_rows(q3, w, rows)
    x = gen(m, k, seed=2).to(torch.bfloat16)
    y = q3.q3_gemm(w, x)
    some = [0, 1, 4000, m - 1]
    xs = x[some].contiguous()
    w64 = h64(q3.q3_gemm(part, torch.eye(k, dtype=torch.bfloat16, device="cuda"))).T
    tol = k * 2.0 ** -23 * (np.abs(h64(xs)) @ np.abs(w64.T))
    assert (np.abs(h64(y[some][:, -rows:]) - h64(xs) @ w64.T) <= tol).all()
    del y
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    dy[:, -rows:] = gen(m, rows, seed=3).to(torch.bfloat16)
    dx = q3.q3_gemm_backward(w, dy)
    d64 = h64(dy[some][:, -rows:])
    tol = n * 2.0 ** -23 * (np.abs(d64) @ np.abs(w64))
    assert (np.abs(h64(dx[some]) - d64 @ w64) <= tol).all()
    del dx
    # the gated block reads gate rows and, half the matrix on, up rows
    h, pre = q3.q3_glu(w, x, save_pre=True)
    assert (np.abs(h64(pre[some][:, -rows:]) - h64(xs) @ w64.T) <= k * 2.0 ** -23 *
            (np.abs(h64(xs)) @ np.abs(w64.T))).all()
    g, u = h64(pre[some][:, n // 2 - rows:n // 2]), h64(pre[some][:, -rows:])
    want = blk.act("silu", g) * u
    assert (np.abs(h64(h[some][:, -rows:]) - want) <= (BF + 2.0 ** -19) * np.abs(want) + 1e-30).all()
    dpre = q3.q3_glu_backward(pre, pre[:, :n // 2], dpre=dy)
    want = blk.glu_backward(h64(pre[[m - 1]]), h64(pre[[m - 1], :n // 2]), "silu")
    assert (np.abs(h64(dpre[[m - 1], -rows:]) - want[:, -rows:]) <= (BF + 2.0 ** -19) * np.abs(want[:, -rows:])).all()


def test_rows_past_32_bits(q3):
    # norms and the sampler on 9.8 GB of rows: the last ones as they come out alone
    m, n = 300_000, 8192
    r = torch.empty(m, n, device="cuda").normal_()
    w = gen(n, seed=1)
    r1, x = q3.q3_residual_norm(r, w, r, w)
    tail = r[-8:].contiguous()
    r2, x2 = q3.q3_residual_norm(tail, w, tail, w)
    assert torch.equal(r1[-8:], r2) and torch.equal(x[-8:], x2)
    del r1, x
    back = q3.q3_residual_norm_backward(r, w, r, r, r, w)
    alone = q3.q3_residual_norm_backward(tail, w, tail, tail, tail, w)
    assert torch.equal(back.dr[-8:], alone.dr) and torch.equal(back.dy[-8:], alone.dy)
    del back
    logits = r.view(-1)[:60_000 * 40_960].view(60_000, 40_960)
    u = torch.rand(60_000, device="cuda")
    tok, lp = q3.q3_sample(logits, u, top_p=torch.full_like(u, 0.5))
    tok2, lp2 = q3.q3_sample(logits[-5:].contiguous(), u[-5:].contiguous(), top_p=torch.full((5,), 0.5, device="cuda"))
    assert torch.equal(tok[-5:], tok2) and torch.equal(lp[-5:], lp2)

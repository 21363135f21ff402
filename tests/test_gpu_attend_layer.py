"""The attention sublayer and the log probabilities run together with the products,
norms and the sampler, as a verify round, a decoding loop and a training step use
them: every stage against 64 bits from what the stage before it gave, captured
graphs, streams, threads and shared workspaces.

Bounds: a product's k 2^-23 sum|x w|; the operators' as in their own tests."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import oracle
import synth
import test_gpu_attend as attend_tests
import test_gpu_logprobs as logprob_tests
import test_gpu_rope as rope_tests
from conftest import ROOT
from gpu_util import pack_layer
from oracle import q3_attend as att
from paged_util import BF, Paged, cuda, host

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


def gen(*shape, seed, scale=1.0, base=0.0):
    return (base + scale * torch.randn(*shape, generator=torch.Generator().manual_seed(seed))).cuda()


def ints(*shape, seed, high):
    return torch.randint(0, high, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()


class Matrix:
    def __init__(self, q3, n, k, seed):
        layer = synth.make_layer(n, k, seed=seed)
        self.w, self.w64 = pack_layer(q3, layer), oracle.dequantize(layer.codes, layer.scales, layer.codebook)


class Layer:
    """Packed qkv, output, gate_up and down matrices and the norms' weights."""

    def __init__(self, q3, k, hq, hk, d, inter, seed):
        self.hq, self.hk, self.d = hq, hk, d
        self.qkv, self.out = Matrix(q3, (hq + 2 * hk) * d, k, seed), Matrix(q3, k, hq * d, seed + 1)
        self.gu, self.dn = Matrix(q3, 2 * inter, k, seed + 2), Matrix(q3, k, inter, seed + 3)
        self.norm, self.ffn_norm = (gen(k, seed=seed + i, scale=0.2, base=1.0) for i in (4, 5))
        self.wq, self.wk = (gen(d, seed=seed + i, scale=0.2, base=1.0) for i in (6, 7))
        self.freq = cuda((1e4 ** (-np.arange(d // 2) * 2 / d)).astype(np.float32))


def attention(q3, layer, r, cache, batch, window=0, keep=None):
    """r -> r + the attention sublayer of r."""
    _, x = q3.q3_residual_norm(r, layer.norm)
    qkv = q3.q3_gemm(layer.qkv.w, x)
    q, _, _ = q3.q3_qk_norm_rope(qkv, layer.hq, layer.hk, layer.freq, None, layer.wq, layer.wk, cache=cache,
                                 batch=batch)
    a, lse = q3.q3_paged_attention(q, cache, batch, window=window, want_lse=True)
    y = q3.q3_gemm(layer.out.w, a)
    if keep is not None:
        keep.append((x, qkv, q, a, lse, y))
    return q3.q3_residual_norm(r, None, y, want_x=False)[0]


def verify(q3, layers, head, final, r, caches, batch, drafts, u, window=0, keep=None):
    """Rows of drafted tokens -> their log probabilities under the model, and tokens drawn from it."""
    for i, (layer, cache) in enumerate(zip(layers, caches)):
        last = i == len(layers) - 1
        r = attention(q3, layer, r, cache, batch, window, keep)
        r, x = q3.q3_ffn(layer.gu.w, layer.dn.w, r, layer.ffn_norm, next_weight=final if last else None, want_x=last)
    logits = q3.q3_gemm(head.w, x)
    lp = q3.q3_logprobs(logits, drafts, 0.7, 5)
    tok, tlp = q3.q3_sample(logits, u, temperature=torch.full_like(u, 0.7))
    return r, logits, lp, tok, tlp


def product_bound(x, w64):
    return x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w64.T)) + 1e-38


@pytest.mark.parametrize("new,length,window", [
    ([1], [77], 0), ([5, 5, 5], [40, 5, 133], 0), ([1, 90, 0, 8], [300, 90, 7, 200], 50), ([260], [300], 0)])
def test_verify_round_stage_by_stage(q3, new, length, window):
    k, hq, hk, d, n = 160, 6, 2, 64, 1000
    layers = [Layer(q3, k, hq, hk, d, 96, seed) for seed in (0, 20)]
    head, final = Matrix(q3, n, k, 50), gen(k, seed=51, scale=0.2, base=1.0)
    rng = np.random.default_rng(5)
    paged = [Paged(rng, new, length, hk, d, 16) for _ in layers]
    paged[1].table = paged[0].table
    for p in paged:
        p.on_device(q3)
    batch, m = paged[0].batch, paged[0].m
    r, drafts, u = gen(m, k, seed=1).bfloat16(), ints(m, seed=2, high=n), torch.rand(m, device="cuda")
    keep = []
    _, logits, lp, tok, tlp = verify(q3, layers, head, final, r, [p.cache for p in paged], batch, drafts, u, window,
                                     keep)
    where = att.places(paged[0].start, paged[0].length, m)
    for layer, p, (x, qkv, q, a, lse, y) in zip(layers, paged, keep):
        assert (np.abs(host(qkv) - host(x) @ layer.qkv.w64.T) <= product_bound(host(x), layer.qkv.w64)).all()
        heads = rope_tests._heads(host(qkv), hq, hk, d)
        wq, wk, freq = host(layer.wq), host(layer.wk), host(layer.freq)
        pos = where[:, 1].astype(np.float64)
        ref = att.head_norm_rope(heads[0], wq, pos, freq, EPS)
        rope_tests._check(q, ref, rope_tests._near(heads[0], wq), "q")
        ref, near = att.head_norm_rope(heads[1], wk, pos, freq, EPS), rope_tests._near(heads[1], wk)
        for i, (s, at) in enumerate(where):
            page, place = att.find(p.table, p.k.shape[0], 16, s, at)
            rope_tests._check(p.cache.k[page, :, place], ref[i], near[i], ("k", i))
            assert torch.equal(p.cache.v[page, :, place], qkv[i].view(-1, d)[hq + hk:].bfloat16())
        p.k, p.v = p.cache.k.cpu(), p.cache.v.cpu()       # what the attention has read
        attend_tests._check(p, q, a, lse, d ** -0.5, window)
        assert (np.abs(host(y) - host(a) @ layer.out.w64.T) <= product_bound(host(a), layer.out.w64)).all()
    l64 = host(logits)
    # the same draw without its log probability: target = the token drawn
    own = q3.q3_logprobs(logits, tok, 0.7)
    t = float(np.float32(0.7))
    for i in range(m):
        want, h, ids, tops = att.logprobs(l64[i], int(drafts[i]), t, 5)
        off = logprob_tests._off(n, want)
        assert abs(float(lp.logprobs[i]) - want) <= off
        assert (host(lp.top_ids)[i] == ids).all()
        assert (np.abs(host(lp.top_logprobs)[i] - tops) <= logprob_tests._off(n, tops)).all()
        drawn = float(att.log_softmax(l64[i], t)[int(tok[i])])
        # the sampler's: fp32 rounding of the result and its fixed-point sum
        assert abs(float(own.logprobs[i]) - float(tlp[i])) <= \
            logprob_tests._off(n, drawn) + 2.0 ** -23 * abs(drawn) + 2e-7


def test_decoding_reads_what_prompts_wrote(q3):
    """A prompt in two chunks, then single tokens: each token's keys and values are those
    that one call over all of them writes, and its attention is the oracle's."""
    hq, hk, d, n = 6, 3, 80, 150
    rng = np.random.default_rng(9)
    whole = Paged(rng, [n], [n], hk, d, 16, stale=float("nan"))
    whole.on_device(q3)
    qkv, freq = gen(n, (hq + 2 * hk) * d, seed=3), cuda((1e4 ** (-np.arange(20) / 20)).astype(np.float32))
    w = gen(d, seed=4, scale=0.2, base=1.0)
    q, _, _ = q3.q3_qk_norm_rope(qkv, hq, hk, freq, None, w, w, interleaved=True, cache=whole.cache,
                                 batch=whole.batch)
    piece = q3.PagedCache(torch.full_like(whole.cache.k, float("nan")), torch.full_like(whole.cache.v, float("nan")))
    at, outs, lses = 0, [], []
    for size in [70, 41] + [1] * (n - 111):
        start, length = cuda(np.array([0, size], np.int32)), cuda(np.array([at + size], np.int32))
        batch = q3.PagedBatch(start, length, cuda(whole.table))
        part, _, _ = q3.q3_qk_norm_rope(qkv[at:at + size], hq, hk, freq, None, w, w, interleaved=True, cache=piece,
                                        batch=batch)
        assert torch.equal(part, q[at:at + size])
        a, l = q3.q3_paged_attention(part, piece, batch, want_lse=True)
        outs.append(a)
        lses.append(l)
        at += size
    live = ~whole.cache.k.isnan()
    assert torch.equal(whole.cache.k[live], piece.k[live]) and torch.equal(whole.cache.v[live], piece.v[live])
    whole.k, whole.v = piece.k.cpu(), piece.v.cpu()
    attend_tests._check(whole, q, torch.cat(outs), torch.cat(lses), d ** -0.5, 0)


def flat(results):
    r, logits, lp, tok, tlp = results
    return [r, logits, lp.logprobs, lp.entropy, lp.stats, lp.top_ids, lp.top_logprobs, tok, tlp]


@pytest.mark.parametrize("new,length", [([4, 4], [300, 41]), ([1] * 3, [20, 500, 64]), ([150, 1], [200, 90])])
def test_captured_rounds_follow_their_inputs(q3, new, length):
    """Two graphs over caches of their own, replayed on two streams at once, with new
    rows and longer sequences; the eager round after each."""
    k, hq, hk, d, n = 96, 4, 2, 64, 500
    layers = [Layer(q3, k, hq, hk, d, 64, seed) for seed in (0, 20)]
    head, final = Matrix(q3, n, k, 50), gen(k, seed=51, scale=0.2, base=1.0)
    sides = []
    for j in range(2):
        rng = np.random.default_rng(60 + j)
        paged = [Paged(rng, new, [x + 40 for x in length], hk, d, 16) for _ in layers]
        for p in paged:
            p.table = paged[0].table
            p.on_device(q3)
        batch, m = paged[0].batch, paged[0].m
        batch.kv_len.copy_(cuda(np.array(length, np.int32)))
        sides.append([gen(m, k, seed=j), [p.cache for p in paged], batch, ints(m, seed=j, high=n),
                      torch.rand(m, device="cuda")])
    def run(s):
        return flat(verify(q3, layers, head, final, *s))
    for s in sides:
        run(s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sides]
    for i in range(4):
        for j, s in enumerate(sides):
            s[0].copy_(gen(s[0].shape[0], k, seed=100 + 2 * i + j))
            s[2].kv_len.add_(3 * i)
            s[3].copy_(ints(s[0].shape[0], seed=200 + 2 * i + j, high=n))
        torch.cuda.synchronize()
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for s, out in zip(sides, outs):
            got = [t.clone() for t in out]
            for a, b in zip(got, run(s)):
                assert torch.equal(a, b)
        torch.zeros(1000, device="cuda").sum().item()


def test_graphs_in_turn_share_a_workspace(q3):
    # one workspace for calls of different kinds and sizes, dirty before each
    rng = np.random.default_rng(3)
    cases = []
    for new, length, hq, hk, d in (([1] * 4, [900, 3, 70, 333], 8, 2, 128), ([200], [700], 4, 1, 64),
                                   ([8, 8], [2000, 500], 16, 2, 128)):
        p = Paged(rng, new, length, hk, d, 16)
        p.on_device(q3)
        cases.append((p, attend_tests._q(rng, p.m, hq, d)))
    logits, targets = gen(2, 90000, seed=1), ints(2, seed=2, high=90000)
    need = max([q3.q3_paged_attention_workspace_bytes(p.m, len(p.new), q.shape[1] // p.dim, p.heads, p.dim)
                for p, q in cases] + [q3.q3_logprobs_workspace_bytes(2, 90000, 7)])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    def run(w):
        out = []
        for p, q in cases:
            out += q3.q3_paged_attention(q, p.cache, p.batch, want_lse=True, workspace=w)
            r = q3.q3_logprobs(logits, targets, 1.0, 7, workspace=w)
            out += [r.logprobs, r.entropy, r.stats, r.top_ids, r.top_logprobs]
        return out
    want = [t.clone() for t in run(None)]
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(ws))
        graphs.append(g)
    for _ in range(4):
        ws.random_(0, 256)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(run(ws), want))


def gradients(q3, layer, qkv, pos, dq, dk, dv, logits, targets, dlp, dh, head):
    """The captured part of a training step: score and its gradient, qkv rows and theirs."""
    q, k, v = q3.q3_qk_norm_rope(qkv, layer.hq, layer.hk, layer.freq, pos, layer.wq, layer.wk)
    g = q3.q3_qk_norm_rope_backward(qkv, layer.hq, layer.hk, layer.freq, pos, dq, dk, dv, layer.wq, layer.wk)
    dx = q3.q3_gemm_backward(layer.qkv.w, g.dqkv)
    lp = q3.q3_logprobs(logits, targets, 0.9)
    dl = q3.q3_logprobs_backward(logits, targets, lp.stats, dlp, dh, 0.9)
    return [q, k, v, g.dqkv, g.dq_weight, g.dk_weight, dx, lp.logprobs, lp.entropy, dl,
            q3.q3_gemm_backward(head.w, dl)]


def test_captured_training_step_beside_an_eager_one(q3):
    k, hq, hk, d, n, m = 96, 4, 2, 64, 496, 70
    layer, head = Layer(q3, k, hq, hk, d, 64, 7), Matrix(q3, n, k, 50)
    ins = [[gen(m, (hq + 2 * hk) * d, seed=10 * j), ints(m, seed=j, high=5000), gen(m, hq * d, seed=10 * j + 1),
            gen(m, hk * d, seed=10 * j + 2), gen(m, hk * d, seed=10 * j + 3), gen(m, n, seed=10 * j + 4),
            ints(m, seed=10 * j + 5, high=n), gen(m, seed=10 * j + 6), gen(m, seed=10 * j + 7)] for j in range(2)]
    eager = gradients(q3, layer, *ins[0], head)
    graphs, outs = [], []
    for s in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gradients(q3, layer, *s, head))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ins]
    for i in range(3):
        for j, s in enumerate(ins):
            s[0].copy_(gen(*s[0].shape, seed=90 + 2 * i + j))
            s[5].copy_(gen(*s[5].shape, seed=190 + 2 * i + j))
        torch.cuda.synchronize()
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
        torch.cuda.synchronize()
        for s, out in zip(ins, outs):
            for a, b in zip(out, gradients(q3, layer, *s, head)):
                assert torch.equal(a, b)
        torch.zeros(1000, device="cuda").sum().item()
    assert all(torch.isfinite(t).all() for t in eager)


class Turned(torch.autograd.Function):
    """The identity, whose gradient is off by a relative amount (a rounding on the way back)."""

    @staticmethod
    def forward(ctx, x, off):
        ctx.save_for_backward(off)
        return x.view_as(x)

    @staticmethod
    def backward(ctx, g):
        return g * (1 + ctx.saved_tensors[0]), None


def plain_heads(x, w, pos, freq):
    """Normed and rotated heads [m][heads][d] in fp64."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a = (pos[:, None] * freq)[:, None]
    h = freq.shape[0]
    lo, hi = x[..., :h], x[..., h:]
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def plain_attention(q, k, v):
    """A causal attention of m tokens in fp64: the caller's own, whose gradient it has too."""
    m, hq, d = q.shape
    k, v = (t.repeat_interleave(hq // t.shape[1], 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
    s = s.masked_fill(torch.ones(m, m, dtype=torch.bool).triu(1), float("-inf"))
    return torch.einsum("hij,jhd->ihd", s.softmax(-1), v).reshape(m, hq * d)


def plain_norm(v, w):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w


@pytest.mark.parametrize("m", [3, 70])
def test_training_step_against_formula_and_differences(q3, m):
    """loss = sum(dlp logprob + dh entropy) of given tokens, through the vocabulary, the
    last norm, the output product, an attention of the caller's, the heads' norms and
    rotation and the qkv product: gradients of r and of every norm's weight."""
    k, hq, hk, d, n = 96, 4, 2, 32, 208
    layer, head = Layer(q3, k, hq, hk, d, 64, 7), Matrix(q3, n, k, 50)
    c = lambda t: t.double().cpu()  # noqa: E731
    r, final, pos = gen(m, k, seed=1), gen(k, seed=2, scale=0.2, base=1.0), ints(m, seed=3, high=3000)
    targets, dlp, dh, temp = ints(m, seed=4, high=n), gen(m, seed=5), gen(m, seed=6, scale=0.3), 1.25
    # forward
    _, x = q3.q3_residual_norm(r, layer.norm)
    qkv = q3.q3_gemm(layer.qkv.w, x)
    q, kk, v = q3.q3_qk_norm_rope(qkv, hq, hk, layer.freq, pos, layer.wq, layer.wk)
    mine = [c(t).view(m, -1, d).requires_grad_() for t in (q, kk, v)]
    a = plain_attention(*mine)
    y = q3.q3_gemm(layer.out.w, a.detach().bfloat16().cuda())
    r1, x1 = q3.q3_residual_norm(r, final, y)
    logits = q3.q3_gemm(head.w, x1)
    lp = q3.q3_logprobs(logits, targets, temp)
    # backward
    dl = q3.q3_logprobs_backward(logits, targets, lp.stats, dlp, dh, temp)
    last = q3.q3_residual_norm_backward(r1, final, q3.q3_gemm_backward(head.w, dl), None, y)
    da = q3.q3_gemm_backward(layer.out.w, last.dy)
    dq, dk, dv = (g.reshape(m, -1).float().cuda() for g in torch.autograd.grad(a, mine, c(da)))
    g = q3.q3_qk_norm_rope_backward(qkv, hq, hk, layer.freq, pos, dq, dk, dv, layer.wq, layer.wk)
    first = q3.q3_residual_norm_backward(r, layer.norm, q3.q3_gemm_backward(layer.qkv.w, g.dqkv), last.dr)
    got = {"r": first.dr, "norm": first.dpre_weight, "final": last.dpre_weight, "wq": g.dq_weight, "wk": g.dk_weight}

    w_qkv, w_out, w_head = (torch.tensor(t.w64) for t in (layer.qkv, layer.out, head))
    p64, f64 = c(pos), c(layer.freq)
    at = {"r": c(r), "norm": c(layer.norm), "final": c(final), "wq": c(layer.wq), "wk": c(layer.wk)}

    def run(w, off):
        x = plain_norm(w["r"], w["norm"]) * (1 + off[0])
        rows = Turned.apply(x @ w_qkv.T, off[1]).view(m, hq + 2 * hk, d)
        q = plain_heads(rows[:, :hq], w["wq"], p64, f64) * (1 + off[2])
        k = plain_heads(rows[:, hq:hq + hk], w["wk"], p64, f64) * (1 + off[3])
        v = rows[:, hq + hk:] * (1 + off[4])
        y = Turned.apply((plain_attention(q, k, v) * (1 + off[5])) @ w_out.T, off[6])
        x1 = plain_norm(w["r"] + y, w["final"]) * (1 + off[7])
        z = torch.log_softmax(Turned.apply(x1 @ w_head.T, off[8]) / temp, 1)
        mine = z.gather(1, targets.cpu().long()[:, None])[:, 0]
        return (c(dlp) * mine).sum() - (c(dh) * (z.exp() * z).sum(1)).sum()

    shapes = [(m, k), (m, (hq + 2 * hk) * d), (m, hq, d), (m, hk, d), (m, hk, d), (m, hq * d), (m, k), (m, k), (m, n)]
    off = [torch.zeros(s, dtype=torch.float64, requires_grad=True) for s in shapes]
    leaves = {name: t.clone().requires_grad_() for name, t in at.items()}
    grads = dict(zip(leaves, torch.autograd.grad(run(leaves, off), list(leaves.values()), create_graph=True)))
    none = [torch.zeros(s, dtype=torch.float64) for s in shapes]
    for name, want in grads.items():
        for seed in range(3):
            way = torch.randn(want.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
            along, e = (want * way).sum(), 1e-6
            up, down = (run(dict(at, **{name: at[name] + s * way}), none) for s in (e, -e))
            assert abs(along.item() - ((up - down) / (2 * e)).item()) <= 1e-5 * (1 + abs(along.item()))
            # first order: 2^-8 for each rounding; a tenth more for the second order and fp32
            carried = sum(t.abs().sum().item() for t in torch.autograd.grad(along, off, retain_graph=True,
                                                                            allow_unused=True) if t is not None)
            fp32 = 2.0 ** -16 * (want.abs() * way.abs()).sum().item()
            assert abs((c(got[name]) * way).sum().item() - along.item()) <= 1.1 * BF * carried + fp32, (name, seed)


def test_threads_on_streams_of_their_own(q3):
    def work(seed):
        rng = np.random.default_rng(seed)
        sets = []
        for new, length, hq, hk, d in (([1] * 3, [700, 30, 64], 8, 2, 128), ([140, 1], [300, 50], 4, 2, 64)):
            p = Paged(rng, new, length, hk, d, 16)
            p.on_device(q3)
            sets.append((p, gen(p.m, (hq + 2 * hk) * d, seed=seed), hq, hk))
        freq = gen(32, seed=seed).abs()
        logits, targets, g = gen(3, 70000, seed=seed), ints(3, seed=seed, high=70000), gen(3, seed=seed)

        def step():
            out = []
            for p, qkv, hq, hk in sets:
                q, _, _ = q3.q3_qk_norm_rope(qkv, hq, hk, freq, cache=p.cache, batch=p.batch)
                out += [q, *q3.q3_paged_attention(q, p.cache, p.batch, want_lse=True)]
                b = q3.q3_qk_norm_rope_backward(qkv, hq, hk, freq, torch.arange(p.m, dtype=torch.int32, device="cuda"),
                                                dq=q, q_weight=torch.ones(p.dim, device="cuda"))
                out += [b.dqkv, b.dq_weight]
            r = q3.q3_logprobs(logits, targets, 1.0, 9)
            return out + [r.logprobs, r.top_ids, q3.q3_logprobs_backward(logits, targets, r.stats, g, g)]
        return step

    steps = [work(s) for s in range(4)]
    want = [[t.clone() for t in s()] for s in steps]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = steps[i]()
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


CHILD = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
import bit_fp8_codebook_amd as q3
from paged_util import Paged
rng = np.random.default_rng(1)
sets = []
for new, length, hq, hk, d in (([1] * 3, [700, 30, 64], 8, 2, 128), ([9, 3], [300, 500], 8, 2, 256), ([300], [400], 4, 1, 192),
                               ([260, 1], [300, 50], 4, 2, 128), ([50], [90], 2, 2, 64)):
    p = Paged(rng, new, length, hk, d, 16)
    p.on_device(q3)
    sets.append((p, torch.randn(p.m, (hq + 2 * hk) * d, device="cuda"), hq, hk))
freq, logits = torch.rand(32, device="cuda"), torch.randn(2, 50000, device="cuda")
targets, g = torch.tensor([5, 49999], dtype=torch.int32, device="cuda"), torch.randn(2, device="cuda")
def step():
    out = []
    for p, qkv, hq, hk in sets:
        q, _, _ = q3.q3_qk_norm_rope(qkv, hq, hk, freq, cache=p.cache, batch=p.batch)
        out += [q, *q3.q3_paged_attention(q, p.cache, p.batch, want_lse=True)]
    r = q3.q3_logprobs(logits, targets, 1.0, 9)
    return out + [r.logprobs, r.top_ids, q3.q3_logprobs_backward(logits, targets, r.stats, g, g)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):      # the library's first call of all
    outs = step()
for i in range(3):
    for _, qkv, _, _ in sets:
        qkv.normal_()
    logits.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip([o.clone() for o in outs], step())), i
    torch.zeros(1000, device="cuda").sum().item()
print("same")
"""


def test_first_call_inside_a_capture(q3):
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"))],
                       env=dict(os.environ), cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-1000:] + r.stderr[-2000:]

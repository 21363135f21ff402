"""The operators between and behind the packed products, as measurable cases.

Five operators of the q3 library, each with a plain form in elementary torch
operations, an evaluation in 64 bits and the work it cannot do without:

  sample   the choice of a token from the vocabulary projection's logits, with
           temperature, top-k, top-p and min-p and given random numbers
  norm     residual_norm: the norm behind a block, its gate, residual scale and
           sum, and the norm before the next block; with back=True its backward
  glu      the gated feed-forward block on packed 3-bit weights (both
           projections, the activation, the product); with step=True the
           gradient of its pre-activations
  linear   the product of many tokens with a packed 3-bit matrix and the
           gradient of its input
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One request's decode step on a 32000-entry vocabulary: the smallest call, latency alone.
        dict(name="sample 1x32000", op="sample", m=1, n=32000, mode="mixed", spread=2.5),
        # An odd vocabulary and an odd batch, each row with its own settings, some with masked (-inf) entries.
        dict(name="sample 33x50257 mixed", op="sample", m=33, n=50257, mode="mixed", spread=2.0),
        # A full batch with plain nucleus sampling at temperature 1: the whole row carries weight.
        dict(name="sample 64x151936 top-p", op="sample", m=64, n=151936, mode="top_p", spread=1.5),
        # One decoded token between two blocks: the latency of the norm in a decode step.
        dict(name="norm 1x4096", op="norm", m=1, n=4096, bf16=True, post=True, gate="none", back=False),
        # A long prompt, fp32 residual stream, a gate of its own for each token.
        dict(name="norm 8192x8192", op="norm", m=8192, n=8192, bf16=False, post=True, gate="full", back=False),
        # Training, bf16 residual stream, per-channel gate shared by all tokens, odd token count.
        dict(name="norm back 2047x5120", op="norm", m=2047, n=5120, bf16=True, post=True, gate="row", back=True),
        # Training, fp32 residual stream, a gate of its own for each token: the largest.
        dict(name="norm back 8192x8192", op="norm", m=8192, n=8192, bf16=False, post=True, gate="full", back=True),
        # A decode step's feed-forward: one token against both projections.
        dict(name="glu 1x14336x4096", op="glu", m=1, i=14336, k=4096, act="silu", step=False),
        # A full verify batch of 64 tokens, tanh-GELU gate.
        dict(name="glu 64x14336x4096", op="glu", m=64, i=14336, k=4096, act="gelu", step=False),
        # A training batch of odd length: pre-activations kept, their gradients returned.
        dict(name="glu step 2000x11008x4096", op="glu", m=2000, i=11008, k=4096, act="silu", step=True),
        # A short prompt through the down projection and back (frozen weights, adapters in front).
        dict(name="linear step 300x4096x14336", op="linear", m=300, n=4096, k=14336),
        # A long prompt through a square projection and back: matrix-core bound.
        dict(name="linear step 4096x8192x8192", op="linear", m=4096, n=8192, k=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "norm", "glu", "linear"])
    if op == "sample":
        n = _log(rng, 100, 200000)
        m = min(_log(rng, 1, 256), max(1, 64 * 151936 // n))
        return dict(op=op, m=m, n=n, mode=rng.choice(["mixed", "mixed", "top_p", "top_k", "min_p", "plain"]),
                    spread=round(rng.uniform(0.5, 4.0), 2))
    if op == "norm":
        n = _log(rng, 64, 12288)
        m = min(_log(rng, 1, 8192), 8192 * 8192 // n)
        return dict(op=op, m=m, n=n, bf16=rng.random() < 0.5, post=rng.random() < 0.7,
                    gate=rng.choice(["none", "row", "full"]), back=rng.random() < 0.5)
    if op == "glu":
        i = 32 * _log(rng, 2, 448)
        k = 32 * _log(rng, 2, 256)
        m = min(_log(rng, 1, 4096), max(1, 2000 * 11008 * 4096 // (i * k)))
        return dict(op=op, m=m, i=i, k=k, act=rng.choice(["silu", "gelu"]), step=rng.random() < 0.5)
    n = _log(rng, 17, 16384)
    k = 32 * _log(rng, 2, 512)
    m = min(_log(rng, 1, 4096), max(1, 4096 * 8192 * 8192 // (n * k)))
    return dict(op=op, m=m, n=n, k=k)


def work(case):
    m = case["m"]
    if case["op"] == "sample":
        # Each logit read once; the row settings and the answers are a few words.
        n = case["n"]
        return {"bytes": 4 * m * n + 28 * m, "flops": 4 * m * n}
    if case["op"] == "norm":
        n, e = case["n"], 2 if case["bf16"] else 4
        gate = {"none": 0, "row": 4 * n, "full": 4 * m * n}[case["gate"]]
        if case["back"]:   # y, r', the gate, dx and dr' in; dr, dy and the gradients of gate and weights out
            return {"bytes": m * n * (4 + e + 4 + e + e + 2) + 2 * gate + 16 * n, "flops": 24 * m * n}
        return {"bytes": m * n * (4 + e + e + 2) + gate + 8 * n, "flops": 12 * m * n}   # y, r -> r', x
    if case["op"] == "glu":
        i, k = case["i"], case["k"]
        b = 2 * i * k * 13 // 32 + 16 * i + 2 * m * k + 2 * m * i
        if case["step"]:
            b += 8 * m * i + 8 * m * i + 4 * m * i + 4 * m * i   # pre out and in, dh in, dpre out
        return {"bytes": b, "flops": 4 * m * i * k}
    n, k = case["n"], case["k"]
    return {"bytes": 2 * (n * k * 13 // 32 + 8 * n) + 2 * m * k + 4 * m * n + 2 * m * n + 4 * m * k,
            "flops": 4 * m * n * k}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _packed(g, n, k):
    """A packed matrix of trained-looking weights: random codes, a bell-shaped
    8-entry codebook for each row, group scales around 2^-6; padding zero."""
    tiles, groups = (n + 15) // 16, k // 32
    gp = 4 * ((groups + 3) // 4)
    code = torch.randint(0, 256, (tiles, 192 * gp), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(119, 123, (tiles, 16 * gp), generator=g, device="cuda", dtype=torch.uint8)
    # Zero what belongs to no row and to no group.
    s = gp // 16
    rows = torch.arange(tiles * 16, device="cuda").reshape(tiles, 1, 1, 1, 16, 1) < n
    live = torch.arange(gp, device="cuda") < groups
    full = code[:, :3072 * s].view(torch.int32).view(tiles, s, 3, 4, 16, 4)
    full *= rows & live[:16 * s].view(1, s, 1, 4, 1, 4)
    fs = scale[:, :256 * s].view(tiles, s, 4, 16, 4)
    fs *= (rows & live[:16 * s].view(1, s, 1, 4, 1, 4))[:, :, 0]
    q = gp % 16 // 4
    if q:
        last = code[:, 3072 * s:].view(torch.int32).view(tiles, 3, q, 16, 4)
        last *= rows[:, 0] & live[16 * s:].view(1, 1, q, 1, 4)
        ls = scale[:, 256 * s:].view(tiles, q, 16, 4)
        ls *= rows[:, 0, 0] & live[16 * s:].view(1, q, 1, 4)
    base = torch.tensor([-1.75, -1.0, -0.55, -0.17, 0.17, 0.55, 1.0, 1.75], device="cuda")
    book = base * (1 + 0.08 * _randn(g, n, 8))
    return dict(n=n, k=k, code=code.view(-1), scale=scale.view(-1),
                book=book.to(torch.float8_e4m3fn).view(torch.uint8).contiguous())


def _pitched(t, to=8):
    """The same values with rows that start at multiples of `to` elements."""
    n = t.shape[1]
    wide = torch.zeros(t.shape[0], (n + to - 1) // to * to, dtype=t.dtype, device=t.device)
    wide[:, :n] = t
    return wide[:, :n]


def prepare(case, seed):
    g = _gen(seed)
    m = case["m"]
    st = dict(case)
    if case["op"] == "sample":
        n, mode = case["n"], case["mode"]
        st["logits"] = _randn(g, m, n) * case["spread"] + 3.0 * (_rand(g, m, n) < 8.0 / n)
        st["u"] = _rand(g, m)
        st["temperature"] = st["top_k"] = st["top_p"] = st["min_p"] = None
        if mode in ("mixed", "top_k", "min_p"):
            st["temperature"] = 0.5 + _rand(g, m)
        if mode in ("mixed", "top_k"):
            st["top_k"] = torch.randint(1, min(n, 200) + 1, (m,), generator=g, device="cuda", dtype=torch.int32)
        if mode in ("mixed", "top_p"):
            st["top_p"] = 0.5 + 0.49 * _rand(g, m)
        if mode in ("mixed", "min_p"):
            st["min_p"] = 0.2 * _rand(g, m) ** 2
        if mode == "mixed":   # each row with its own subset of the settings, some greedy
            off = _rand(g, 4, m)
            st["temperature"][off[0] < 0.15] = 0.0
            st["top_k"][off[1] < 0.4] = 0
            st["top_p"][off[2] < 0.4] = 1.0
            st["min_p"][off[3] < 0.5] = 0.0
        if mode in ("mixed", "top_k"):   # a grammar's or a ban list's mask on some rows
            banned = (_rand(g, m, n) < 0.3) & (_rand(g, m, 1) < 0.4)
            st["logits"].masked_fill_(banned, -math.inf)
        return st
    if case["op"] == "norm":
        n, t = case["n"], torch.bfloat16 if case["bf16"] else torch.float32
        st["y"] = _randn(g, m, n) * 0.7
        st["r"] = (_randn(g, m, n) * (1 + 4 * (_rand(g, 1, n) < 0.01))).to(t)
        st["pre_weight"] = 1 + 0.2 * _randn(g, n)
        st["post_weight"] = 1 + 0.2 * _randn(g, n) if case["post"] else None
        st["gate"] = {"none": lambda: None, "row": lambda: 0.5 * _randn(g, n),
                      "full": lambda: 0.5 * _randn(g, m, n)}[case["gate"]]()
        st["rscale"] = 0.75
        if case["back"]:   # r is then the sum that the forward kept
            st["dx"] = _randn(g, m, n)
            st["dr"] = _randn(g, m, n).to(t)
        return st
    n = 2 * case["i"] if case["op"] == "glu" else case["n"]
    st["w"] = _packed(g, n, case["k"])
    st["x"] = (_randn(g, m, case["k"]) * (1 + 4 * (_rand(g, 1, case["k"]) < 0.01))).to(torch.bfloat16)
    if case["op"] == "glu" and case["step"]:
        st["dh"] = _randn(g, m, case["i"])
    if case["op"] == "linear":
        st["dy"] = _pitched(_randn(g, m, n).to(torch.bfloat16))
    return st


# ------------------------------------------------------------------ plain forms

def _weights(w):
    """The packed matrix as float32 [n][k]."""
    n, k = w["n"], w["k"]
    tiles, groups = (n + 15) // 16, k // 32
    gp = 4 * ((groups + 3) // 4)
    s, q = gp // 16, gp % 16 // 4
    words = w["code"].view(tiles, 192 * gp)
    scales = w["scale"].view(tiles, 16 * gp)
    # [tile][row][group][word]
    d = words[:, :3072 * s].view(torch.int32).view(tiles, s, 3, 4, 16, 4).permute(0, 4, 1, 3, 5, 2).reshape(
        tiles * 16, 16 * s, 3)
    e = scales[:, :256 * s].view(tiles, s, 4, 16, 4).permute(0, 3, 1, 2, 4).reshape(tiles * 16, 16 * s)
    if q:
        d2 = words[:, 3072 * s:].view(torch.int32).view(tiles, 3, q, 16, 4).permute(0, 3, 2, 4, 1).reshape(
            tiles * 16, 4 * q, 3)
        e2 = scales[:, 256 * s:].view(tiles, q, 16, 4).permute(0, 2, 1, 3).reshape(tiles * 16, 4 * q)
        d, e = torch.cat([d, d2], 1), torch.cat([e, e2], 1)
    b = d[:n, :groups].contiguous().view(torch.uint8).view(n, groups, 3, 4)
    low, mid, top = b & 7, (b >> 3) & 7, b >> 6
    spare = top[:, :, 0] | top[:, :, 1] << 2 | top[:, :, 2] << 4
    codes = torch.cat([torch.stack([low, mid], 3).view(n, groups, 24), spare & 7, spare >> 3], 2).view(n, k)
    book = w["book"].view(torch.float8_e4m3fn).float()
    return (torch.gather(book, 1, codes.long()).view(n, groups, 32)
            * torch.exp2(e[:n, :groups].float() - 127).unsqueeze(2)).view(n, k)


def _plain_sample(st):
    logits = st["logits"]
    m, n = logits.shape
    one = torch.ones(m, 1, device="cuda", dtype=torch.float64)

    def setting(name, default):
        return one * default if st[name] is None else st[name].double().view(m, 1)

    temp, top_k = setting("temperature", 1.0), setting("top_k", 0)
    top_p, min_p = setting("top_p", 1.0), setting("min_p", 0.0)
    greedy = temp <= 0
    sl, order = torch.sort(logits, dim=1, descending=True, stable=True)   # equal logits: lower index first
    # 64 bits: the running sums of 151936 weights decide between neighbours.
    sl = sl.double()
    w = torch.exp((sl - sl[:, :1]) / torch.where(greedy, one, temp))
    rank = torch.arange(n, device="cuda").view(1, n)
    kept = torch.where((top_k > 0) & (top_k < n), rank < top_k, rank >= 0) & (w > 0)
    kept &= torch.where(greedy, rank < 1, rank >= 0)
    w = w * kept
    before = torch.cumsum(w, 1) - w
    kept &= (top_p >= 1) | (before < top_p * w.sum(1, keepdim=True)) | (rank == 0)
    kept &= w >= min_p
    w = w * kept
    p = torch.zeros_like(w).scatter_(1, order, w)   # back in index order
    run = torch.cumsum(p, 1)
    total = run[:, -1:]
    token = ((run > st["u"].double().view(m, 1) * total) & (p > 0)).to(torch.int8).argmax(1, keepdim=True)
    logprob = torch.log(torch.gather(p, 1, token) / total)
    return token.view(m).int(), logprob.view(m).float()


def _plain_norm(st):
    y, r = st["y"], st["r"].float()
    t = y
    if st["post"]:
        t = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * st["post_weight"]
    if st["gate"] is not None:
        t = t * st["gate"]
    out = r + st["rscale"] * t
    x = out * torch.rsqrt((out * out).mean(1, keepdim=True) + EPS) * st["pre_weight"]
    return out.to(st["r"].dtype), x.to(torch.bfloat16)


def _plain_norm_back(st):
    out, y, scale = st["r"].float(), st["y"], st["rscale"]
    s = torch.rsqrt((out * out).mean(1, keepdim=True) + EPS)
    hat = out * s
    a = st["dx"] * st["pre_weight"]
    grad = st["dr"].float() + s * (a - hat * (a * hat).mean(1, keepdim=True))
    res = {"dr": grad.to(st["r"].dtype), "dpre_weight": (st["dx"] * hat).sum(0)}
    dt = scale * grad if st["gate"] is None else scale * grad * st["gate"]
    if st["post"]:
        sy = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        yh = y * sy
        t = yh * st["post_weight"]
        b = dt * st["post_weight"]
        res["dpost_weight"] = (dt * yh).sum(0)
        res["dy"] = (sy * (b - yh * (b * yh).mean(1, keepdim=True))).to(torch.bfloat16)
    else:
        t = y
        res["dy"] = dt.to(torch.bfloat16)
    if st["gate"] is not None:
        dg = scale * grad * t
        res["dgate"] = dg.sum(0) if st["gate"].dim() == 1 else dg
    return res


def _act(act, z):
    """The activation and its derivative."""
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _plain_glu(st):
    i = st["i"]
    pre = st["x"].float() @ _weights(st["w"]).t()
    a, da = _act(st["act"], pre[:, :i])
    h = (a * pre[:, i:]).to(torch.bfloat16)
    if not st["step"]:
        return h
    dpre = torch.cat([st["dh"] * pre[:, i:] * da, st["dh"] * a], 1).to(torch.bfloat16)
    return {"h": h, "pre": pre, "dpre": dpre}


def _plain_linear(st):
    w = _weights(st["w"])
    return {"y": st["x"].float() @ w.t(), "dx": st["dy"].float() @ w}


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _own(st)
    if st["op"] == "sample":
        return _plain_sample(st)
    if st["op"] == "norm":
        return _plain_norm_back(st) if st["back"] else _plain_norm(st)
    return _plain_glu(st) if st["op"] == "glu" else _plain_linear(st)


def _own(st):
    import bit_fp8_codebook_amd as q3
    op = st["op"]
    if op == "sample":
        return q3.q3_sample(st["logits"], st["u"], st["temperature"], st["top_k"], st["top_p"], st["min_p"])
    if op == "norm":
        block = dict(y=st["y"], post_weight=st["post_weight"], gate=st["gate"], scale=st["rscale"], eps=EPS)
        if not st["back"]:
            return q3.q3_residual_norm(st["r"], st["pre_weight"], **block)
        g = q3.q3_residual_norm_backward(st["r"], st["pre_weight"], dx=st["dx"], dr_out=st["dr"], **block)
        res = {"dr": g.dr, "dpre_weight": g.dpre_weight, "dy": g.dy}
        if st["post"]:
            res["dpost_weight"] = g.dpost_weight
        if st["gate"] is not None:
            res["dgate"] = g.dgate
        return res
    p = st["w"]
    w = q3.PackedMatrix(p["n"], p["k"], p["code"], p["scale"], p["book"])
    if op == "glu":
        if not st["step"]:
            return q3.q3_glu(w, st["x"], act=st["act"])
        h, pre = q3.q3_glu(w, st["x"], act=st["act"], save_pre=True)
        return {"h": h, "pre": pre, "dpre": q3.q3_glu_backward(pre, st["dh"], act=st["act"])}
    return {"y": q3.q3_gemm(w, st["x"]), "dx": q3.q3_gemm_backward(w, st["dy"])}


# ------------------------------------------------------------------ 64 bits

def _weights64(w):
    """The packed matrix in 64 bits, element by element from the placement rule."""
    n, k = w["n"], w["k"]
    gp = 4 * ((k // 32 + 3) // 4)
    r = torch.arange(n, device="cuda").view(n, 1)
    c = torch.arange(k, device="cuda").view(1, k)
    g, p = c // 32, c % 32
    step, kb, t = g // 16, g % 16 // 4, g % 4
    q = torch.clamp((gp - 16 * step) // 4, max=4)

    def byte(j, lane):
        at = r // 16 * (192 * gp) + 3072 * step + 16 * (16 * (q * j + kb) + r % 16) + 4 * t + lane
        return w["code"][at].int()

    # Weights 0..23: three bits of byte p % 4 of word p // 8; weights 24..31: two bits of each word's byte.
    lane, word = p % 4, torch.clamp(p // 8, max=2)
    code = (byte(word, lane) >> (3 * (p % 8 // 4))) & 7
    spare = sum((byte(j, lane) >> 6) << (2 * j) for j in range(3))
    code = torch.where(p < 24, code, (spare >> (3 * ((p - 24) // 4).clamp(min=0))) & 7)
    entry = w["book"][r.expand(n, k), code.long()].int()
    mag, ex = entry & 7, (entry >> 3) & 15
    v = torch.where(ex == 0, torch.ldexp(mag.double(), torch.full_like(ex, -9)),
                    torch.ldexp(8 + mag.double(), ex - 10))
    v = torch.where(entry >= 128, -v, v)
    e = w["scale"][r // 16 * (16 * gp) + 256 * step + 4 * (16 * kb + r % 16) + t].int()
    return torch.ldexp(v, e - 127)


def _exact_sample(st):
    logits = st["logits"].cpu().numpy().astype(np.float64)
    m, n = logits.shape
    host = {k: None if st[k] is None else st[k].cpu().numpy().astype(np.float64)
            for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    tokens, logprobs = np.zeros(m, np.int32), np.zeros(m, np.float64)
    for i in range(m):
        def setting(name, off):
            return off if host[name] is None else host[name][i]
        row, temp = logits[i], setting("temperature", 1.0)
        if temp <= 0:
            tokens[i] = int(np.argmax(row))
            continue
        order = np.lexsort((np.arange(n), -row))
        if 0 < setting("top_k", 0) < n:
            order = order[:int(setting("top_k", 0))]
        p = np.exp((row[order] - row[order[0]]) / temp)
        if setting("top_p", 1.0) < 1:
            order = order[:max(1, int(np.searchsorted(np.cumsum(p), setting("top_p", 1.0) * p.sum(), side="left")) + 1)]
            p = p[:len(order)]
        order = np.sort(order[p >= setting("min_p", 0.0)])
        p = np.exp((row[order] - row.max()) / temp)
        order, p = order[p > 0], p[p > 0]
        at = min(int(np.searchsorted(np.cumsum(p), host["u"][i] * p.sum(), side="right")), len(order) - 1)
        tokens[i] = order[at]
        logprobs[i] = np.log(p[at]) - np.log(p.sum())
    return tokens, logprobs


def _exact_norm(st):
    y, r, gain = st["y"].double(), st["r"].double(), st["pre_weight"].double()
    n = y.shape[1]
    gate = 1.0 if st["gate"] is None else st["gate"].double()
    ry = (y.pow(2).sum(1, keepdim=True) / n + EPS).pow(-0.5) if st["post"] else 1.0
    pw = st["post_weight"].double() if st["post"] else 1.0
    if not st["back"]:
        out = r + st["rscale"] * gate * pw * (y * ry)
        return out, gain * out * (out.pow(2).sum(1, keepdim=True) / n + EPS).pow(-0.5)
    rx = (r.pow(2).sum(1, keepdim=True) / n + EPS).pow(-0.5)
    dx = st["dx"].double()
    inner = (dx * gain * r).sum(1, keepdim=True)
    grad = st["dr"].double() + rx * gain * dx - rx.pow(3) / n * inner * r
    res = {"dr": grad, "dpre_weight": (dx * r * rx).sum(0)}
    up = st["rscale"] * grad * gate
    if st["post"]:
        res["dpost_weight"] = (up * y * ry).sum(0)
        res["dy"] = ry * pw * up - ry.pow(3) / n * (up * pw * y).sum(1, keepdim=True) * y
    else:
        res["dy"] = up * torch.ones_like(y)
    if st["gate"] is not None:
        dg = st["rscale"] * grad * pw * (y * ry)
        res["dgate"] = dg.sum(0) if st["gate"].dim() == 1 else dg
    return res


def _exact_glu(st):
    i = st["i"]
    w = _weights64(st["w"])
    g, u = st["x"].double() @ w[:i].t(), st["x"].double() @ w[i:].t()
    if st["act"] == "silu":
        a = g / (1 + torch.exp(-g))
        da = (1 + torch.exp(-g) * (1 + g)) / (1 + torch.exp(-g)) ** 2
    else:
        c = math.sqrt(2 / math.pi)
        e = torch.exp(-2 * c * (g + 0.044715 * g ** 3))   # 0.5 (1 + tanh v) = 1 / (1 + exp(-2 v))
        a = g / (1 + e)
        da = 1 / (1 + e) + g * e / (1 + e) ** 2 * 2 * c * (1 + 0.134145 * g ** 2)
        da = torch.where(torch.isfinite(e * e), da, torch.zeros_like(da))
    if not st["step"]:
        return a * u
    dh = st["dh"].double()
    return {"h": a * u, "pre": torch.cat([g, u], 1), "dpre": torch.cat([dh * u * da, dh * a], 1)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(st)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "glu":
        return _exact_glu(st)
    w = _weights64(st["w"])
    return {"y": st["x"].double() @ w.t(), "dx": st["dy"].double() @ w}

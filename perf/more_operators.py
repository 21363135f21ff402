"""The operators of an attention sublayer and of scored tokens, as measurable cases.

Three operators of the q3 library, each with a plain form in elementary torch
operations, an evaluation in 64 bits and the work it cannot do without:

  rope      q3_qk_norm_rope: the norms of each head's query and key and the
            rotation by position, from the qkv product's fp32 rows to bf16 queries
            and to the pages of a cache; with back=True its backward, of plain rows
  attend    q3_paged_attention: new tokens of several sequences (one decoded token,
            a few drafted ones, a chunk of a prompt) over a paged cache
  logprobs  q3_logprobs: log probabilities of given tokens, the entropy and the top
            alternatives of rows of logits; with step=True its gradient too
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One request's decoded token between the qkv product and attention: latency alone.
        dict(name="rope 1x40x128", op="rope", back=False, b=1, n=1, past=4000, page=64, hq=32, hk=8, d=128, rot=128,
             pairs=False, norm=True),
        # Prompts of four requests, ragged, into the cache.
        dict(name="rope 4 prompts x40x128", op="rope", back=False, b=4, n=2048, past=100, page=16, hq=32, hk=8, d=128,
             rot=128, pairs=False, norm=True),
        # Training, an odd token count, adjacent pairs and half of the head rotated.
        dict(name="rope back 4095x80x128", op="rope", back=True, m=4095, hq=64, hk=8, d=128, rot=64, pairs=True,
             norm=True, bf16=True),
        # One request decodes over a short context: latency.
        dict(name="attend 1x1 over 4000", op="attend", b=1, n=1, past=3999, mixed=False, page=64, hq=32, hk=8, d=128,
             window=0),
        # A full batch decodes, contexts of all lengths up to 16384, small pages.
        dict(name="attend 64x1 to 16384", op="attend", b=64, n=1, past=16383, mixed=False, page=16, hq=32, hk=8,
             d=128, window=0),
        # A verify round: eight drafted tokens of four requests with contexts up to 262144.
        dict(name="attend 4x8 to 262144", op="attend", b=4, n=8, past=262136, mixed=False, page=64, hq=64, hk=8, d=128,
             window=0),
        # A chunk of a long prompt: matrix-core bound, the largest.
        dict(name="attend 1x2048 over 32000", op="attend", b=1, n=2048, past=30000, mixed=False, page=128, hq=32, hk=8,
             d=128, window=0),
        # A chunk and eight decoding requests in one batch, three heads to a key, a sliding window.
        dict(name="attend 500 and 8x1 window", op="attend", b=9, n=500, past=4000, mixed=True, page=32, hq=24, hk=8,
             d=64, window=1024),
        # One request's scores on a 32000-entry vocabulary: the smallest call.
        dict(name="logprobs 1x32000 top 20", op="logprobs", step=False, m=1, n=32000, top=20, temperature=1.0,
             masks=False, spread=2.5),
        # A verify round of 64 tokens, masked entries, top alternatives.
        dict(name="logprobs 64x151936 top 20", op="logprobs", step=False, m=64, n=151936, top=20, temperature=0.8,
             masks=True, spread=2.0),
        # A training step on an odd vocabulary with an entropy term, some tokens without a target.
        dict(name="logprobs step 2047x50257", op="logprobs", step=True, m=2047, n=50257, top=0, temperature=1.0,
             masks=True, spread=2.0),
        # The same on a large vocabulary: memory alone.
        dict(name="logprobs step 2048x151936", op="logprobs", step=True, m=2048, n=151936, top=0, temperature=1.0,
             masks=False, spread=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "logprobs"])
    if op == "logprobs":
        n = _log(rng, 100, 200000)
        step = rng.random() < 0.5
        m = min(_log(rng, 1, 4096), max(1, 2048 * 151936 // n))
        return dict(op=op, step=step, m=m, n=n, top=0 if step else rng.choice([0, 1, 5, 20, 32]),
                    temperature=rng.choice([1.0, 0.7, 1.3]), masks=rng.random() < 0.5,
                    spread=round(rng.uniform(0.5, 4.0), 2))
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "rope":
        rot = rng.choice([d, d, d // 2])
        most = max(1, 8192 * 40 * 128 // ((hq + 2 * hk) * d))
        case = dict(op=op, back=rng.random() < 0.5, hq=hq, hk=hk, d=d, rot=rot, pairs=rng.random() < 0.5,
                    norm=rng.random() < 0.8)
        if case["back"]:
            return dict(case, m=min(_log(rng, 1, 8192), most), bf16=rng.random() < 0.5)
        b = min(_log(rng, 1, 64), most)
        return dict(case, b=b, n=min(_log(rng, 1, 8192), max(1, most // b)), past=_log(rng, 1, 4096) - 1, page=page)
    kind = rng.choice(["decode", "verify", "chunk", "mixed"])
    b = {"decode": _log(rng, 1, 128), "verify": _log(rng, 1, 32), "chunk": _log(rng, 1, 4),
         "mixed": _log(rng, 2, 16)}[kind]
    n = {"decode": 1, "verify": rng.randint(2, 16), "chunk": _log(rng, 64, 2048), "mixed": _log(rng, 16, 512)}[kind]
    # No more cache than 4 x 262144 x 8 x 128, no more pairs than the largest listed case has.
    most = min(4 * 262144 * 8 * 128 // (b * hk * d), 2048 * 32 * 32048 * 128 // (b * n * hq * d), 262144)
    past = _log(rng, 1, max(1, most - n))
    return dict(op=op, b=b, n=n, past=past, mixed=kind == "mixed", page=page, hq=hq, hk=hk, d=d,
                window=rng.choice([0, 0, _log(rng, 16, 4096)]))


def _spread(lo, hi, b, phase):
    """b whole numbers from lo to hi, the first hi, the others all over the range."""
    return [hi] + [lo + int((hi - lo + 1) * ((i * 0.6180339887498949 + phase) % 1.0)) for i in range(1, b)]


def _lengths(case):
    """New tokens and whole length (those included) of each sequence."""
    b, n, past = case["b"], case["n"], case["past"]
    new = [n] + [1] * (b - 1) if case.get("mixed") else _spread(n if n < 16 else max(1, n // 4), n, b, 0.3)
    return new, [p + t for p, t in zip(_spread(past // 8, past, b, 0.0), new)]


def _pairs(t, length, window):
    """Visible (query, key) pairs of t new tokens at the end of a sequence."""
    if not window:
        return t * length - t * (t - 1) // 2
    return sum(min(window, p + 1) for p in range(length - t, length))


def work(case):
    if case["op"] == "logprobs":
        m, n = case["m"], case["n"]
        if case["step"]:   # the logits once, their gradients once
            return {"bytes": 6 * m * n + 24 * m, "flops": 12 * m * n}
        return {"bytes": 4 * m * n + 12 * m + 8 * m * case["top"], "flops": 6 * m * n}
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "rope":
        if case["back"]:   # the qkv rows and the three gradients in, the rows' gradient out
            e = case["m"] * (hq + 2 * hk) * d
            return {"bytes": e * (4 + (2 if case["bf16"] else 4) + 2), "flops": 14 * e}
        e = sum(_lengths(case)[0]) * (hq + 2 * hk) * d
        return {"bytes": 6 * e, "flops": 8 * e}
    new, whole = _lengths(case)
    w = case["window"]
    seen = [min(k, w + t - 1) if w else k for t, k in zip(new, whole)]
    return {"bytes": sum(seen) * hk * d * 4 + sum(new) * hq * (4 * d + 4),
            "flops": 4 * hq * d * sum(_pairs(t, k, w) for t, k in zip(new, whole))}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _paged(case, g):
    """A cache in pages, in no order, and the sequences' tables; what no sequence holds is stale."""
    new, whole = _lengths(case)
    page, b = case["page"], case["b"]
    held = [(k + page - 1) // page for k in whole]
    pages = sum(held) + 3
    shape = (pages, case["hk"], page, case["d"])
    table = np.full((b, max(held)), -1, np.int32)
    ids = torch.randperm(pages, generator=g, device="cuda").cpu().numpy()
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = ids[at:at + h]
        at += h
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(k=torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16),
                v=torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16), table=dev(table),
                start=dev(np.concatenate([[0], np.cumsum(new)])), length=dev(whole), m=sum(new), most=max(new))


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "logprobs":
        m, n = case["m"], case["n"]
        st["logits"] = _randn(g, m, n).mul_(case["spread"])
        hot = torch.randint(0, n, (m, 1), generator=g, device="cuda")   # a few likely tokens a row
        hot = (hot + torch.arange(8, device="cuda") * (n // 8)) % n
        st["logits"].scatter_add_(1, hot, 4 + 2 * _randn(g, m, 8))
        st["targets"] = torch.where(_rand(g, m) < 0.7, hot[:, 0],
                                    torch.randint(0, n, (m,), generator=g, device="cuda")).int()
        if case["masks"]:   # a ban list on some rows, tokens without a target (-1)
            for rows in torch.split(torch.arange(m, device="cuda"), 256):
                banned = (_rand(g, len(rows), n) < 0.2) & (_rand(g, len(rows), 1) < 0.4)
                st["logits"][rows] = st["logits"][rows].masked_fill(banned, -math.inf)
            st["targets"] = torch.where(_rand(g, m) < 0.1, -1, st["targets"]).int()
        if case["step"]:
            st["dlogprobs"] = -_rand(g, m) / m
            st["dentropy"] = 0.01 * _randn(g, m) / m
        return st
    hq, hk, d = case["hq"], case["hk"], case["d"]
    if case["op"] == "attend":
        st["cache"] = _paged(case, g)
        st["q"] = (1.5 * _randn(g, st["cache"]["m"], hq * d)).to(torch.bfloat16)
        return st
    st["freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda").double() / case["rot"])).float()
    st["wq"] = 1 + 0.2 * _randn(g, d) if case["norm"] else None
    st["wk"] = 1 + 0.2 * _randn(g, d) if case["norm"] else None
    if not case["back"]:
        st["cache"] = _paged(case, g)
        st["qkv"] = _randn(g, st["cache"]["m"], (hq + 2 * hk) * d)
        return st
    m, t = case["m"], torch.bfloat16 if case["bf16"] else torch.float32
    st["qkv"] = _randn(g, m, (hq + 2 * hk) * d)
    # Packed documents: each starts again at 0, or goes on from far away.
    st["positions"] = (torch.arange(m, device="cuda") % 1021 + 100000 * (torch.arange(m, device="cuda") // 1021 % 2)).int()
    st["dq"], st["dk"], st["dv"] = (_randn(g, m, h * d).to(t) for h in (hq, hk, hk))
    return st


# ------------------------------------------------------------------ plain forms

def _places(c):
    """Sequence, place among its new tokens and position of each token."""
    i = torch.arange(c["m"], device="cuda")
    s = (i.view(-1, 1) >= c["start"][1:].view(1, -1)).sum(1)
    t = i - c["start"][s]
    return s, t, c["length"][s] - (c["start"][s + 1] - c["start"][s]) + t


def _turn(x, freq, positions, pairs, back=False):
    """The first 2 len(freq) values of each head of x [m][heads][d] rotated."""
    angle = positions.double().view(-1, 1, 1) * freq.double()   # far positions need 64 bits
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    if back:
        s = -s
    r = 2 * len(freq)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    u, v = a * c - b * s, b * c + a * s
    turned = torch.stack([u, v], -1).flatten(-2) if pairs else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rope(st):
    hq, hk, d, c = st["hq"], st["hk"], st["d"], st["cache"]
    x = st["qkv"].view(c["m"], hq + 2 * hk, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if st["norm"]:
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * st["wq"]
        k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS) * st["wk"]
    s, _, position = _places(c)
    q = _turn(q, st["freq"], position, st["pairs"])
    k = _turn(k, st["freq"], position, st["pairs"])
    page, at = c["table"][s, position // st["page"]].long(), position % st["page"]
    c["k"][page, :, at] = k.to(torch.bfloat16)
    c["v"][page, :, at] = v.to(torch.bfloat16)
    return {"q": q.to(torch.bfloat16).view(c["m"], hq * d), "k": c["k"], "v": c["v"]}


def _plain_rope_back(st):
    m, hq, hk, d = st["m"], st["hq"], st["hk"], st["d"]
    x = st["qkv"].view(m, hq + 2 * hk, d)
    q, k = x[:, :hq], x[:, hq:hq + hk]
    gq = _turn(st["dq"].float().view(m, hq, d), st["freq"], st["positions"], st["pairs"], True)
    gk = _turn(st["dk"].float().view(m, hk, d), st["freq"], st["positions"], st["pairs"], True)
    res = {}
    if st["norm"]:
        sq = torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS)
        sk = torch.rsqrt((k * k).mean(-1, keepdim=True) + EPS)
        res["dq_weight"], res["dk_weight"] = (gq * q * sq).sum((0, 1)), (gk * k * sk).sum((0, 1))
        gq, gk = gq * st["wq"], gk * st["wk"]
        gq = sq * (gq - q * sq * (gq * q * sq).mean(-1, keepdim=True))
        gk = sk * (gk - k * sk * (gk * k * sk).mean(-1, keepdim=True))
    res["dqkv"] = torch.cat([gq, gk, st["dv"].float().view(m, hk, d)], 1).view(m, -1).to(torch.bfloat16)
    return res


def _plain_attend(st):
    hq, hk, d, c = st["hq"], st["hk"], st["d"], st["cache"]
    b, n, group = st["b"], c["most"], hq // hk
    s, t, _ = _places(c)
    i = torch.arange(n, device="cuda")
    new = c["start"][1:] - c["start"][:-1]
    # Padded to the most new tokens and the longest sequence: [b][kv head][head of it][token]
    q = st["q"][(c["start"][:-1].view(b, 1) + i).clamp(max=c["m"] - 1)].float()
    q = q.view(b, n, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b * hk, group * n, d)
    pages = c["table"].clamp(min=0).long()
    keys = c["k"][pages].transpose(1, 2).reshape(b * hk, -1, d).float()
    score = torch.bmm(q, keys.transpose(1, 2).contiguous()).mul_(1 / math.sqrt(d)).view(b, hk, group, n, -1)
    del keys
    position = (c["length"] - new).view(b, 1) + i
    j = torch.arange(score.shape[-1], device="cuda")
    seen = j <= position.unsqueeze(2)
    if st["window"]:
        seen &= j > position.unsqueeze(2) - st["window"]
    score.masked_fill_(~seen.view(b, 1, 1, n, -1), -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    values = c["v"][pages].transpose(1, 2).reshape(b * hk, -1, d).float()
    out = torch.bmm(weight.view(b * hk, group * n, -1), values).view(b, hk, group, n, d) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(b, n, hq * d)[s, t].to(torch.bfloat16)
    lse = (top + torch.log(total)).permute(0, 3, 1, 2, 4).reshape(b, n, hq)[s, t]
    return {"out": out, "lse": lse}


def _plain_logprobs(st):
    logits, m, n = st["logits"], st["m"], st["n"]
    z = logits / st["temperature"]
    z -= z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    zp = torch.where(e > 0, z, torch.zeros_like(z))
    entropy = torch.log(total) - (e * zp).sum(1, keepdim=True) / total
    some = (st["targets"] >= 0).view(m, 1)
    target = st["targets"].clamp(min=0).long().view(m, 1)
    log_total = torch.log(total)
    logprob = torch.where(some, torch.gather(z, 1, target) - log_total, torch.zeros_like(total))
    res = {"logprobs": logprob.view(m), "entropy": entropy.view(m)}
    if st["top"]:
        best, order = torch.sort(logits, dim=1, descending=True, stable=True)   # equal logits: lower index first
        best, order = best[:, :st["top"]], order[:, :st["top"]]
        res["top_ids"] = torch.where(best > -math.inf, order, -1).int()
        res["top_logprobs"] = (best - best[:, :1]) / st["temperature"] - log_total
    if st["step"]:
        p = e / total
        given = torch.where(some.view(m), st["dlogprobs"], 0.0).view(m, 1)
        dz = -p * (given + st["dentropy"].view(m, 1) * (zp - log_total + entropy))
        live = torch.gather(e, 1, target) > 0
        dz.scatter_add_(1, target, torch.where(live, given, torch.zeros_like(given)))
        res["dlogits"] = (dz / st["temperature"]).to(torch.bfloat16)
    return res


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _own(st)
    if st["op"] == "rope":
        return _plain_rope_back(st) if st["back"] else _plain_rope(st)
    return _plain_attend(st) if st["op"] == "attend" else _plain_logprobs(st)


def _own(st):
    import bit_fp8_codebook_amd as q3
    if st["op"] == "logprobs":
        r = q3.q3_logprobs(st["logits"], st["targets"], temperature=st["temperature"], top=st["top"])
        res = {"logprobs": r.logprobs, "entropy": r.entropy}
        if st["top"]:
            res["top_ids"], res["top_logprobs"] = r.top_ids, r.top_logprobs
        if st["step"]:
            res["dlogits"] = q3.q3_logprobs_backward(st["logits"], st["targets"], r.stats, st["dlogprobs"],
                                                     st["dentropy"], temperature=st["temperature"])
        return res
    if st["op"] == "rope" and st["back"]:
        g = q3.q3_qk_norm_rope_backward(st["qkv"], st["hq"], st["hk"], st["freq"], st["positions"], st["dq"], st["dk"],
                                        st["dv"], q_weight=st["wq"], k_weight=st["wk"], eps=EPS,
                                        interleaved=st["pairs"])
        res = {"dq_weight": g.dq_weight, "dk_weight": g.dk_weight} if st["norm"] else {}
        return dict(res, dqkv=g.dqkv)
    c = st["cache"]
    cache, batch = q3.PagedCache(c["k"], c["v"]), q3.PagedBatch(c["start"], c["length"], c["table"])
    if st["op"] == "rope":
        q, _, _ = q3.q3_qk_norm_rope(st["qkv"], st["hq"], st["hk"], st["freq"], q_weight=st["wq"], k_weight=st["wk"],
                                     eps=EPS, interleaved=st["pairs"], cache=cache, batch=batch)
        return {"q": q, "k": c["k"], "v": c["v"]}
    out, lse = q3.q3_paged_attention(st["q"], cache, batch, window=st["window"], want_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ 64 bits

def _exact_turn(x, freq, positions, pairs, sign):
    """Each pair as a complex number times e^(i angle)."""
    r = 2 * len(freq)
    angle = sign * positions.double()[:, None] * freq.double()[None, :]
    z = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    y = x.clone()
    if pairs:
        y[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)) * z).flatten(-2)
    else:
        w = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * z
        y[..., :r // 2], y[..., r // 2:r] = w.real, w.imag
    return y


def _exact_rope(st):
    hq, hk, d, c = st["hq"], st["hk"], st["d"], st["cache"]
    new, whole = _lengths(st)
    positions = torch.cat([torch.arange(k - t, k, device="cuda") for t, k in zip(new, whole)])
    q, k, v = st["qkv"].double().split([hq * d, hk * d, hk * d], 1)

    def head(x, w):
        x = x.reshape(c["m"], -1, d)
        if w is not None:
            x = x * w.double() / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        return _exact_turn(x, st["freq"], positions, st["pairs"], 1)
    q, k, v = head(q, st["wq"]), head(k, st["wk"]), v.reshape(c["m"], hk, d)
    ck, cv, table = c["k"].double(), c["v"].double(), c["table"].cpu().tolist()
    at = 0
    for s, (t, length) in enumerate(zip(new, whole)):
        place = torch.arange(length - t, length)
        page = torch.tensor(table[s])[place // st["page"]].cuda()
        inside = (place % st["page"]).cuda()
        ck[page, :, inside], cv[page, :, inside] = k[at:at + t], v[at:at + t]
        at += t
    return {"q": q.reshape(c["m"], hq * d), "k": ck, "v": cv}


def _exact_rope_back(st):
    m, hq, hk, d = st["m"], st["hq"], st["hk"], st["d"]
    q, k, _ = st["qkv"].double().split([hq * d, hk * d, hk * d], 1)
    res = {}

    def head(x, g, w, name):
        x, g = x.reshape(m, -1, d), g.double().reshape(m, -1, d)
        g = _exact_turn(g, st["freq"], st["positions"], st["pairs"], -1)
        if w is None:
            return g.reshape(m, -1)
        root = (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
        res[name] = (g * x / root).sum((0, 1))
        g = g * w.double()
        return (g / root - x * (g * x).sum(-1, keepdim=True) / (d * root.pow(3))).reshape(m, -1)
    gq, gk = head(q, st["dq"], st["wq"], "dq_weight"), head(k, st["dk"], st["wk"], "dk_weight")
    return dict(res, dqkv=torch.cat([gq, gk, st["dv"].double()], 1))


def _exact_attend(st):
    hq, hk, d, c, page = st["hq"], st["hk"], st["d"], st["cache"], st["page"]
    new, whole = _lengths(st)
    out = torch.empty(c["m"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(c["m"], hq, dtype=torch.float64, device="cuda")
    at = 0
    for s, (t, length) in enumerate(zip(new, whole)):
        pages = c["table"][s, :(length + page - 1) // page].long()
        p = torch.arange(length - t, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hidden = (j > p) | (j <= p - st["window"]) if st["window"] else j > p
        for h in range(hk):
            keys = c["k"][pages, h].reshape(-1, d)[:length].double()
            values = c["v"][pages, h].reshape(-1, d)[:length].double()
            for i in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = st["q"][at:at + t, i * d:(i + 1) * d].double() @ keys.t() / math.sqrt(d)
                score[hidden] = -math.inf
                lse[at:at + t, i] = torch.logsumexp(score, 1)
                out[at:at + t, i] = torch.softmax(score, 1) @ values
        at += t
    return {"out": out.reshape(c["m"], hq * d), "lse": lse}


def _exact_logprobs(st):
    m, n, top = st["m"], st["n"], st["top"]
    res = {"logprobs": torch.zeros(m, dtype=torch.float64, device="cuda"),
           "entropy": torch.zeros(m, dtype=torch.float64, device="cuda")}
    if top:
        res["top_ids"] = np.full((m, top), -1, np.int32)
        res["top_logprobs"] = torch.full((m, top), -math.inf, dtype=torch.float64, device="cuda")
    if st["step"]:
        res["dlogits"] = torch.empty(m, n, dtype=torch.float64, device="cuda")
    for rows in torch.split(torch.arange(m), 256):
        a, b = int(rows[0]), int(rows[-1]) + 1
        logp = torch.log_softmax(st["logits"][a:b].double() / st["temperature"], 1)
        p = torch.exp(logp)
        log0 = torch.where(p > 0, logp, torch.zeros_like(logp))
        entropy = -(p * log0).sum(1)
        res["entropy"][a:b] = entropy
        chosen = torch.zeros_like(p)
        for i, t in enumerate(st["targets"][a:b].tolist()):
            if t >= 0:
                res["logprobs"][a + i] = logp[i, t]
                chosen[i, t] = 1.0
            if top:
                row = st["logits"][a + i].cpu().numpy()
                best = np.lexsort((np.arange(n), -row))[:top]
                best = best[row[best] > -np.inf]
                res["top_ids"][a + i, :len(best)] = best
                res["top_logprobs"][a + i, :len(best)] = logp[i, torch.from_numpy(best).cuda()]
        if st["step"]:
            g = st["dlogprobs"][a:b].double()[:, None]
            first = g * (chosen * (p > 0) - p * chosen.sum(1, keepdim=True))
            second = st["dentropy"][a:b].double()[:, None] * -p * (log0 + entropy[:, None])
            res["dlogits"][a:b] = (first + second) / st["temperature"]
    return res


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(st)
    if case["op"] == "attend":
        return _exact_attend(st)
    return _exact_rope_back(st) if case["back"] else _exact_rope(st)

"""Batches over a paged cache for the GPU tests, made on the host."""
import numpy as np
import torch

BF = 2.0 ** -8     # half a step of bfloat16, relative
F32 = 2.0 ** -24


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().double().cpu().numpy()


class Paged:
    """Sequences of `new` tokens at the end of `length` positions, in pages of no
    order; what no sequence holds is `stale`."""

    def __init__(self, rng, new, length, heads, dim, page, spare=2, stale=0.0, wide=0, gap=0):
        self.new, self.length, self.page, self.heads, self.dim = list(new), list(length), page, heads, dim
        held = [(n + page - 1) // page for n in self.length]
        pages = sum(held) + spare
        self.table = np.full((len(new), max(max(held), 1) + wide), -1, np.int32)
        ids = rng.permutation(pages)
        at = 0
        for s, h in enumerate(held):
            self.table[s, :h] = ids[at:at + h]
            at += h
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.m = int(self.start[-1])
        shape = (pages, heads, page, dim)
        self.k = torch.from_numpy(rng.normal(size=shape)).to(torch.bfloat16)
        self.v = torch.from_numpy(rng.normal(size=shape)).to(torch.bfloat16)
        live = np.zeros((pages, page), bool)
        for s, n in enumerate(self.length):
            for p in range(n):
                live[self.table[s, p // page], p % page] = True
        dead = torch.from_numpy(~live)[:, None, :, None].expand(shape)
        self.k[dead] = stale
        self.v[dead] = stale
        self.gap = gap

    def on_device(self, q3):
        """(cache, batch); with a gap the pages lie apart."""
        n = self.heads * self.page * self.dim
        def place(t):
            wide = torch.full((t.shape[0], n + self.gap), float("nan"), dtype=t.dtype)
            wide[:, :n] = t.reshape(t.shape[0], n)
            wide = wide.cuda()
            return wide.as_strided(t.shape, (n + self.gap, self.page * self.dim, self.dim, 1))
        self.cache = q3.PagedCache(place(self.k), place(self.v))
        self.batch = q3.PagedBatch(cuda(self.start), cuda(np.array(self.length, np.int32)), cuda(self.table))
        return self.cache, self.batch

"""q3_paged_attention on inputs in which one lost, repeated or misplaced key shows,
over every kernel form, parts of a row and lists of pages that are made again.

Counting: queries of zeros give every key the weight 1, so that lse is the logarithm
of a whole number below 2^24, summed without rounding.  Picking: a row's query has
one key whose weight is 1 beside weights of e^-64, so that the row's output is that
key's value, to the bit."""
import math

import pytest
import torch

from paged_util import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_fp8_codebook_amd as q3
    q3.lib()
    return q3


class Batch:
    """Sequences of `new` tokens at the end of `length` positions in pages of no order;
    shared: all of them read one sequence's pages (the longest's)."""

    def __init__(self, q3, new, length, hq, hk, d, page, window, shared=False, seed=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        held = [(n + page - 1) // page for n in length]
        pages = (max(held) if shared else sum(held)) + 2
        ids = torch.randperm(pages, generator=g, device="cuda").int()
        self.table = torch.full((len(new), max(held)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for s, h in enumerate(held):
            self.table[s, :h] = ids[at:at + h]
            at += 0 if shared else h
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        start = [sum(new[:s]) for s in range(len(new) + 1)]
        self.m, self.hq, self.hk, self.d, self.page, self.window = start[-1], hq, hk, d, page, window
        shape = (pages, hk, page, d)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        self.v.copy_(torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.int8))
        self.v.mul_(2).sub_(1)      # 1 and -1
        self.length = length
        self.sequence = torch.repeat_interleave(torch.arange(len(new), device="cuda"),
                                                torch.tensor(new, device="cuda"))
        row = torch.arange(self.m, device="cuda")
        begin, n, whole = (torch.tensor(a, device="cuda") for a in (start[:-1], new, length))
        self.position = (whole - n - begin)[self.sequence] + row
        low = self.position - window + 1 if window else torch.zeros_like(self.position)
        self.seen = self.position - low.clamp(min=0) + 1
        self.cache = q3.PagedCache(self.k, self.v)
        self.batch = q3.PagedBatch(i32(start), i32(length), self.table)
        self.q3 = q3

    def run(self, q, scale):
        return self.q3.q3_paged_attention(q, self.cache, self.batch, scale, self.window, want_lse=True)

    def count_off(self):
        """log2 good to two of its steps, three constants' and products' half steps: 7 half steps of ln n."""
        return 7 * F32 * torch.log(self.seen.double()) + 1e-12

    def check_counts(self):
        q = torch.zeros(self.m, self.hq * self.d, dtype=torch.bfloat16, device="cuda")
        out, lse = self.run(q, 0.125)
        n, off = self.seen.double(), self.count_off()
        assert (off < 0.5 / (n + 1)).all()      # a key more or less would show
        assert ((lse.double() - torch.log(n)[:, None]).abs() <= off[:, None]).all()
        # and the values, whole sums: the rows of the first and the last few tokens
        group = self.hq // self.hk
        for t in {0, 1, self.m // 2, self.m - 1} & set(range(self.m)):
            s, p, c = int(self.sequence[t]), int(self.position[t]), int(self.seen[t])
            at = torch.arange(p - c + 1, p + 1, device="cuda")
            v = self.v[self.table[s, at // self.page].long(), :, at % self.page].double()
            mean = (v.sum(0) / c).repeat_interleave(group, 0).reshape(-1)
            assert ((out[t].double() - mean).abs() <= 1.01 * (BF + 4 * F32) * mean.abs()).all(), t

    def marks(self, s):
        """Positions of sequence s to be picked, one for each value of a head at most: ends of
        steps, tiles and pages, the last keys of all, and those spread over the sequence."""
        n = self.length[s]
        want = [n - 1, 0, n // 2, 31, 32, 63, 64, 127, 128, self.page - 1, self.page, n - 2, n - 64, n - 65, n - 128, n - 129]
        if self.window:
            want += [n - self.window - 1, n - self.window, n - self.window + 1]
        want += [(i * n // self.d) // 64 * 64 - i % 2 for i in range(1, self.d)]
        return list(dict.fromkeys(p for p in want if 0 <= p < n))[:self.d]

    def check_picks(self, calls=4, shared=False):
        d, hq = self.d, self.hq
        marks = [self.marks(0 if shared else s) for s in range(len(self.length))]
        for s, where in enumerate(marks[:1] if shared else marks):
            at = torch.tensor(where, device="cuda")
            page = self.table[s, at // self.page].long()
            for c in range(0, len(where)):
                self.k[page[c], :, where[c] % self.page, c] = 1
        size = torch.tensor([len(w) for w in marks], device="cuda")
        place = torch.zeros(len(marks), d, dtype=torch.long, device="cuda")
        for s, where in enumerate(marks):
            place[s, :len(where)] = torch.tensor(where, device="cuda")
        r = torch.arange(self.m * hq, device="cuda").view(self.m, hq)
        head = torch.arange(hq, device="cuda") // (hq // self.hk)
        self.v.mul_(1 + torch.rand(self.v.shape, device="cuda", dtype=torch.bfloat16))   # values that tell keys apart
        for call in range(calls):
            pick = (r + call * self.m * hq) % size[self.sequence][:, None]
            q = torch.zeros(self.m, hq, d, dtype=torch.bfloat16, device="cuda")
            q.scatter_(2, pick[:, :, None], 64.0)
            out, lse = self.run(q.view(self.m, hq * d), 1.0)
            at = place[self.sequence[:, None], pick]
            sees = (at <= self.position[:, None]) & (at > (self.position - self.seen)[:, None])
            page = self.table[self.sequence[:, None], at // self.page].long()
            value = self.v[page, head[None, :].expand_as(page), at % self.page]
            assert torch.equal(out.view(self.m, hq, d)[sees], value[sees]), call
            # 64 and what e^-64 adds; the constants' and the products' half steps
            assert ((lse.double() - 64).abs()[sees] <= 64 * 4 * F32).all()
            rest = torch.log(self.seen.double())[:, None].expand(self.m, hq)
            off = self.count_off()[:, None].expand(self.m, hq)
            assert ((lse.double() - rest).abs()[~sees] <= off[~sees]).all()


# new, length, hq, hk, page: few rows a sequence, in tiles of 32 and of 64; many, in one part, a few and many
CASES = {
    "decode": ([1, 1, 1], [70001, 130, 2500], 8, 2, 16),
    "decode, a tile cut many times": ([1], [66000], 3, 1, 64),
    "decode, many short": ([1] * 70, [(67 * i) % 501 + 1 for i in range(70)], 4, 2, 64),
    "verify": ([9, 2, 5], [70001, 130, 2500], 8, 2, 16),
    "verify, a tile cut many times": ([20, 1], [20000, 9000], 3, 1, 32),
    "many parts": ([100, 1, 1], [70001, 130, 2500], 8, 2, 16),
    "several parts": ([200, 3], [3001, 40], 2, 1, 64),
    "two parts": ([600], [5003], 16, 8, 128),
    "one part": ([400], [801], 48, 24, 64),
    "mixed": ([300, 1, 0, 40], [2900, 777, 5, 40], 8, 8, 8),
}


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("d", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("name", CASES)
def test_no_key_is_lost(q3, name, d, window):
    new, length, hq, hk, page = CASES[name]
    b = Batch(q3, new, length, hq, hk, d, page, window)
    b.check_counts()
    b.check_picks()


# More pages than a block lists at a time (2048), in one block's part: pages of 1 and 2
# positions, and the smallest that whole runs are read from, 16 and 32
AGAIN = {
    "decode, pages of 1": ([1] * 64, [5000 + 7 * i for i in range(64)], 16, 8, 1, False),
    "verify, pages of 1": ([9] * 64, [5000 + 7 * i for i in range(64)], 32, 8, 1, False),
    "chunk, pages of 1": ([1600], [6007], 32, 8, 1, False),
    "chunk, pages of 2": ([1600], [9007], 32, 8, 2, False),
    "chunk, pages of 16": ([1601], [40011], 32, 8, 16, False),
    "decode, pages of 32": ([1] * 700, [80000 - i for i in range(700)], 2, 1, 32, True),
    "verify, pages of 32": ([9] * 700, [80000 - 16 * i for i in range(700)], 4, 1, 32, True),
}


@pytest.mark.parametrize("windowed", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("name", AGAIN)
def test_no_key_is_lost_where_pages_are_listed_again(q3, name, d, windowed):
    new, length, hq, hk, page, shared = AGAIN[name]
    # a window that begins inside a step and inside a page, and leaves more pages than a list holds
    window = length[-1] - 237 if windowed else 0
    b = Batch(q3, new, length, hq, hk, d, page, window, shared)
    b.check_counts()
    b.check_picks(2, shared)

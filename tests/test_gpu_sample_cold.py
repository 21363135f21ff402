"""Sampling where most of the row weighs nothing (low temperatures, confident
rows): top-k and min-p borders that fall among entries without weight, on the
GPU against the fp64 oracle, and that such rows cost what others do."""
import statistics

import numpy as np
import pytest
import torch

from test_gpu_sample import check, q3, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1000, 4000, 20481, 50257, 151936])
@pytest.mark.parametrize("t", [1e-4, 0.01, 0.1, 0.3])
def test_borders_among_entries_without_weight(q3, n, t):  # noqa: F811
    l, u = rows(6, n, seed=n)
    l[3] = np.round(l[3])                        # thousands of equal entries at each border
    l[4, ::7] = -np.inf
    l[5, 1:] -= 60.0                             # one entry far above the rest
    temp = [t] * 6
    check(q3, l, u, temp, top_k=[50] * 6)
    check(q3, l, u, temp, top_k=[50] * 6, top_p=[0.9, 0.5, 0.999, 0.9, 0.95, 0.99])
    check(q3, l, u, temp, min_p=[1e-20, 1e-13, 1e-14, 1e-30, 1e-20, 1e-20])
    check(q3, l, u, temp, [2, 5, n - 1, n // 2, 1000, 50], [0.9, 1.0, 0.3, 1.0, 0.9999999, 0.9],
          [1e-20, 0.05, 1e-14, 1e-13, 0.0, 1e-30])


@pytest.mark.parametrize("m,n", [(8, 16000), (8, 151936)])
def test_low_temperatures_cost_what_others_do(q3, m, n):  # noqa: F811
    # a row cut by bisection takes tens of passes over it, ten times these calls' time and more
    g = torch.Generator(device="cuda").manual_seed(0)
    l = 2 * torch.randn(m, n, generator=g, device="cuda")
    u = torch.rand(m, generator=g, device="cuda")
    full = lambda v, t=torch.float32: torch.full((m,), v, dtype=t, device="cuda")  # noqa: E731

    def time(temperature, **kw):
        took = []
        for _ in range(9):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                q3.q3_sample(l, u, full(temperature), **kw)
            b.record()
            torch.cuda.synchronize()
            took.append(a.elapsed_time(b))
        return statistics.median(took)

    k50 = full(50, torch.int32)
    for kw in (dict(top_k=k50), dict(top_k=k50, top_p=full(0.9)), dict(min_p=full(1e-20))):
        warm = time(1.0, **kw)
        for t in (0.1, 0.01):
            assert time(t, **kw) <= 3 * warm, (kw.keys(), t)

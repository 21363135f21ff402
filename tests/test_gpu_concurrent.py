"""Several calls at once: host threads with a stream each, and a first call of the
large-LDS kernels that is already inside a capture (a process of its own)."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import synth
from conftest import ROOT
from gpu_util import pack_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q3():
    import bit_fp8_codebook_amd
    bit_fp8_codebook_amd.lib()
    return bit_fp8_codebook_amd


def rand(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda().to(dtype)


def test_threads_on_streams_of_their_own(q3):
    w = pack_layer(q3, synth.make_layer(1024, 544, seed=1))
    n = 4100

    def work(seed):
        x, r, y = rand(70, 544, seed=seed, dtype=torch.bfloat16), rand(9, n, seed=seed), rand(9, n, seed=seed + 50)
        l, u, wt = rand(3, 40000, seed=seed), rand(3, seed=seed).abs() % 1.0, rand(n, seed=seed)

        def step():
            h, pre = q3.q3_glu(w, x, save_pre=True)
            g = q3.q3_residual_norm_backward(r, wt, y, r, y, wt)
            return (h, pre, q3.q3_gemm(w, x), q3.q3_gemm(w, x[:20]), q3.q3_gemm_backward(w, pre.bfloat16()), g.dr,
                    g.dy, g.dpre_weight, g.dpost_weight, *q3.q3_residual_norm(r, wt, y, wt),
                    *q3.q3_sample(l, u, top_p=u * 0 + 0.9))
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
sys.path[:0] = [{root!r}]
import torch
import bit_fp8_codebook_amd as q3
w = q3.empty_packed(2048, 512, "cuda")
for t, lo, hi in ((w.code_plane, 0, 256), (w.scale_plane, 118, 123), (w.codebook, 0x28, 0x48)):
    t.random_(lo, hi)
x = torch.randn(1600, 512, device="cuda").bfloat16()
r, y, one = torch.randn(40, 12288, device="cuda"), torch.randn(40, 12288, device="cuda"), torch.ones(12288, device="cuda")
def step():
    g = q3.q3_residual_norm_backward(r, one, y, r, y, one)
    return (q3.q3_gemm(w, x), q3.q3_gemm(w, x[:300]), q3.q3_gemm(w, x[:100]), q3.q3_gemm(w, x[:48]),
            *q3.q3_glu(w, x, save_pre=True), q3.q3_glu(w, x[:90]), q3.q3_gemm_backward(w, x.repeat(1, 4)), g.dr, g.dy,
            g.dpre_weight)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):          # the library's first call of all
    outs = step()
for i in range(3):
    x.copy_(torch.randn(1600, 512, device="cuda")); y.normal_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, step())), i
    torch.zeros(1000, device="cuda").sum().item()
print("same")
"""


def test_first_call_inside_a_capture(q3):
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], env=dict(os.environ), cwd=ROOT,
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-1000:] + r.stderr[-2000:]

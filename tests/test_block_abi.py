"""The C ABI of include/q3_block.h without a GPU: every declared entry point is
exported and bound, workspace sizes, and refusals before any HIP call."""
import ctypes
import os
import re
import subprocess

import pytest

from conftest import ROOT

HEADER = os.path.join(ROOT, "include", "q3_block.h")
FAKE = 0x1000   # never dereferenced: every call below fails validation first
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def L():
    from bit_fp8_codebook_amd import _block, _lib
    if not os.path.exists(_lib.LIB_PATH):
        from bit_fp8_codebook_amd import build
        build.build(verbose=False)
    return _block.lib()


def test_header_library_and_binding_agree(L):
    from bit_fp8_codebook_amd import _block, _lib
    declared = set(re.findall(r"Q3_API\s+[\w\s\*]+?\b(q3_\w+)\s*\(", open(HEADER).read()))
    assert declared == set(_block.SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True).stdout
    assert declared <= set(re.findall(r"\bT\s+(q3_\w+)", out))


def test_workspace_sizes(L):
    # up to 64 tokens: the small products' own; more: the widened matrix, k padded to 128 (n to 64 transposed)
    assert L.q3_gemm_workspace_bytes(4096, 4096, 64) == L.q3_gemm_small_m_workspace_bytes(4096, 4096, 64)
    assert L.q3_gemm_workspace_bytes(4096, 96, 4096) == 4096 * 128 * 2
    assert L.q3_glu_workspace_bytes(4096, 96, 64) == 0
    assert L.q3_glu_workspace_bytes(4096, 96, 4096) == 4096 * 128 * 2
    assert L.q3_gemm_backward_workspace_bytes(128, 96, 5) == 96 * 128 * 2
    # a ragged n also keeps dy's rows padded
    assert L.q3_gemm_backward_workspace_bytes(45, 96, 5) == 96 * 64 * 2 + 768
    for f in (L.q3_gemm_workspace_bytes, L.q3_gemm_backward_workspace_bytes, L.q3_glu_workspace_bytes):
        assert f(64, 33, 100) == 0 and f(64, 64, 0) == 0 and f(0, 64, 100) == 0
    assert L.q3_glu_workspace_bytes(96, 64, 100) == 0                    # I not a multiple of 32
    f = L.q3_residual_norm_backward_workspace_bytes
    assert f(1, 64) == 3 * 256 and f(1, 16385) == 0 and f(0, 64) == 0
    assert L.q3_sample_workspace_bytes(0, 10) == 0 and L.q3_sample_workspace_bytes(65536, 10) == 0
    assert L.q3_sample_workspace_bytes(1, (1 << 19) + 1) == 0
    assert L.q3_sample_workspace_bytes(2, 100) > 0


def _mat(n=64, k=64, **kw):
    from bit_fp8_codebook_amd import _lib
    d = dict(code_plane=FAKE, scale_plane=FAKE, codebook=FAKE)
    d.update(kw)
    return _lib.Q3Matrix(n, k, d["code_plane"], d["scale_plane"], d["codebook"])


def test_gemm_refusals(L):
    ws = 1 << 30
    for f, cols in ((L.q3_gemm, 64), (L.q3_gemm_backward, 64)):
        call = lambda w=_mat(), x=FAKE, m=100, ldx=64, y=FAKE, ldy=64, p=FAKE, b=ws: f(  # noqa: E731
            ctypes.byref(w) if w else None, x, m, ldx, y, ldy, p, b, None)
        assert call(w=None) == 1 and call(x=None) == 1 and call(y=None) == 1
        assert call(m=0) == 2 and call(m=-1) == 2 and call(m=1 << 31) == 2
        assert call(ldx=56) == 1 and call(ldy=63) == 1
        assert call(ldx=68) == 3 and call(x=FAKE + 8) == 3 and call(y=FAKE + 2) == 3
        assert call(p=FAKE + 16) == 3 and call(p=None) == 1 and call(b=64) == 1
        assert call(w=_mat(k=48)) == 2 and call(w=_mat(code_plane=FAKE + 4)) == 3
        assert call(w=_mat(code_plane=None)) == 1
        assert call(ldx=1 << 23) == 2                                     # 256 rows pass 32 bits of bytes
    huge = _mat(n=1 << 20, k=8192)
    assert L.q3_gemm(ctypes.byref(huge), FAKE, 100, 8192, FAKE, 1 << 20, FAKE, 1 << 40, None) == 2


def test_glu_refusals(L):
    call = lambda w=_mat(128), x=FAKE, m=100, ldx=64, act=0, h=FAKE, ldh=64, pre=FAKE, ldp=128, p=FAKE, b=1 << 30: \
        L.q3_glu(ctypes.byref(w), x, m, ldx, act, h, ldh, pre, ldp, p, b, None)  # noqa: E731
    assert call(act=2) == 1 and call(act=-1) == 1
    assert call(w=_mat(96)) == 2
    assert call(h=None) == 1 and call(ldh=56) == 1 and call(ldp=124) == 1
    assert call(ldh=68) == 3 and call(h=FAKE + 8) == 3 and call(ldp=130) == 3 and call(pre=FAKE + 4) == 3
    assert call(p=None) == 1 and call(b=100) == 1 and call(p=FAKE + 128) == 3
    assert call(m=0) == 2 and call(x=None) == 1 and call(ldx=60) == 1
    back = lambda pre=FAKE, lp=128, dh=FAKE, ld=64, act=1, m=3, i=64, o=FAKE, lo=128: L.q3_glu_backward(  # noqa: E731
        pre, lp, dh, ld, act, m, i, o, lo, None)
    assert back(pre=None) == 1 and back(dh=None) == 1 and back(o=None) == 1 and back(act=7) == 1
    assert back(lp=124) == 1 and back(ld=60) == 1 and back(lo=120) == 1
    assert back(lp=130) == 3 and back(ld=66) == 3 and back(lo=132) == 3 and back(dh=FAKE + 4) == 3
    assert back(m=0) == 2 and back(i=48) == 2 and back(i=0) == 2


def test_norm_refusals(L):
    def call(y=FAKE, ldy=64, pw=FAKE, g=FAKE, lg=64, r=FAKE, ldr=64, ro=FAKE, ldro=64, t=F32, w=FAKE, x=FAKE, ldx=64,
             eps=1e-6, m=3, n=64):
        return L.q3_residual_norm(y, ldy, pw, g, lg, 1.0, r, ldr, ro, ldro, t, w, x, ldx, eps, m, n, None)
    assert call(t=2) == 1 and call(t=-1) == 1
    assert call(m=0) == 2 and call(n=0) == 2 and call(n=16385) == 2
    assert call(r=None) == 1 and call(ro=None) == 1 and call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(y=None) == 1 and call(y=None, pw=None) == 1 and call(y=None, g=None) == 1   # weights without y
    assert call(x=None) == 1 and call(x=None, w=None, y=None, pw=None, g=None, ro=None) == 1
    assert call(ldy=63) == 1 and call(ldr=63) == 1 and call(ldro=63) == 1 and call(ldx=63) == 1 and call(lg=63) == 1
    assert call(ro=FAKE, ldro=72) == 1                                    # in place with another pitch
    assert call(y=FAKE + 2) == 3 and call(r=FAKE + 2) == 3 and call(x=FAKE + 1) == 3 and call(g=FAKE + 1) == 3
    assert call(r=FAKE + 1, t=BF16) == 3 and call(w=FAKE + 2) == 3 and call(ro=FAKE + 2) == 3


def test_norm_backward_refusals(L):
    from bit_fp8_codebook_amd._block import Q3ResidualNormGrads

    def call(y=FAKE, pw=FAKE, g=FAKE, lg=64, t=F32, ws=FAKE, b=1 << 20, null=False, n=64, **kw):
        d = dict(dx=FAKE, ld_dx=64, dr_out=FAKE, ld_dr_out=64, dr=FAKE, ld_dr=64, dy=FAKE, ld_dy=64, dgate=FAKE,
                 ld_dgate=64, dpost_weight=FAKE, dpre_weight=FAKE)
        d.update(kw)
        gr = Q3ResidualNormGrads(**d)
        return L.q3_residual_norm_backward(y, 64, pw, g, lg, 1.0, FAKE, 64, t, FAKE, 1e-6, 3, n,
                                           None if null else ctypes.byref(gr), ws, b, None)
    assert call(null=True) == 1 and call(dr=None) == 1
    assert call(y=None, pw=None, g=None, dgate=None, dpost_weight=None) == 1      # dy without y
    assert call(g=None) == 1 and call(pw=None) == 1                               # a gradient without its input
    assert call(ld_dx=63) == 1 and call(ld_dr=63, dr_out=None) == 1 and call(ld_dr_out=63) == 1
    assert call(ld_dy=63) == 1 and call(ld_dgate=63) == 1 and call(ld_dr=72) == 1   # dr in place, other pitch
    assert call(dx=FAKE + 2) == 3 and call(dy=FAKE + 1) == 3 and call(dr=FAKE + 2) == 3 and call(dgate=FAKE + 2) == 3
    assert call(ws=None) == 1 and call(b=100) == 1 and call(ws=FAKE + 64) == 3 and call(t=5) == 1 and call(n=0) == 2


def test_sample_refusals(L):
    def call(l=FAKE, m=2, n=100, ld=100, t=FAKE, k=FAKE, p=FAKE, mp=FAKE, u=FAKE, ws=FAKE, b=1 << 30, tok=FAKE, lp=FAKE):
        return L.q3_sample(l, m, n, ld, t, k, p, mp, u, ws, b, tok, lp, None)
    assert call(l=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(m=0) == 2 and call(m=65536) == 2 and call(n=0) == 2 and call(n=(1 << 19) + 1, ld=1 << 20) == 2
    assert call(ld=99) == 1 and call(ws=None) == 1 and call(b=100) == 1
    assert call(l=FAKE + 2) == 3 and call(t=FAKE + 1) == 3 and call(k=FAKE + 2) == 3 and call(ws=FAKE + 128) == 3
    assert call(u=FAKE + 2) == 3 and call(tok=FAKE + 1) == 3 and call(lp=FAKE + 2) == 3


def test_binding_refusals():
    # The binding sees shapes, types and devices before any pointer leaves it.
    import torch
    from bit_fp8_codebook_amd import _block as b
    cpu = torch.device("cpu")
    with pytest.raises(ValueError):
        b._rows(torch.empty(3, 4), (3, 5), torch.float32, cpu, "t")
    with pytest.raises(ValueError):
        b._rows(torch.empty(5, 3).t(), (3, 5), torch.float32, cpu, "t")
    with pytest.raises(ValueError):
        b._rows(torch.empty(3, 5, dtype=torch.float64), (3, 5), torch.float32, cpu, "t")
    with pytest.raises(ValueError):
        b._rows(torch.empty(1, 5).expand(3, 5), (3, 5), torch.float32, cpu, "t")
    with pytest.raises(ValueError):
        b._rows(torch.empty(3, 5, device="meta"), (3, 5), torch.float32, cpu, "t")
    assert b._rows(torch.empty(4, 9)[:3, :5], (3, 5), torch.float32, cpu, "t") is not None
    for bad in (torch.empty(3, 64, dtype=torch.bfloat16), None):
        with pytest.raises(ValueError):
            b._tokens(bad, 64, "x")                                       # not on a device
    with pytest.raises(ValueError):
        b._act("relu")
    with pytest.raises(ValueError):
        b.q3_sample(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(ValueError):
        b.q3_residual_norm(torch.zeros(2, 10))
    with pytest.raises(ValueError):
        b.q3_glu_backward(torch.zeros(2, 64), torch.zeros(2, 32))


def test_ffn_refusals(L):
    from bit_fp8_codebook_amd._block import Q3FfnNorms
    need = L.q3_ffn_workspace_bytes(128, 64, 100)
    assert need == 100 * 64 * 2 + 100 * 64 * 2 + 100 * 64 * 4 + L.q3_glu_workspace_bytes(128, 64, 100)
    assert L.q3_ffn_workspace_bytes(96, 64, 100) == 0 and L.q3_ffn_workspace_bytes(128, 1 << 15, 100) == 0
    assert L.q3_ffn_workspace_bytes(128, 64, 0) == 0 and L.q3_ffn_workspace_bytes(0, 64, 1) == 0

    def call(gu=_mat(128), dn=_mat(64), act=0, null=False, r=FAKE, ldr=64, ro=FAKE, ldro=64, t=F32, x=FAKE, ldx=64, m=100,
             ws=FAKE, b=need, **kw):
        d = dict(pre_weight=FAKE, post_weight=FAKE, next_weight=FAKE, gate=FAKE, ld_gate=64, scale=1.0, eps=1e-6)
        d.update(kw)
        norms = Q3FfnNorms(**d)
        return L.q3_ffn(ctypes.byref(gu) if gu else None, ctypes.byref(dn) if dn else None, act,
                        None if null else ctypes.byref(norms), r, ldr, ro, ldro, t, x, ldx, m, ws, b, None)
    assert call(gu=None) == 1 and call(dn=None) == 1 and call(null=True) == 1 and call(act=2) == 1
    assert call(gu=_mat(96)) == 2 and call(dn=_mat(96)) == 2 and call(dn=_mat(64, 96)) == 2 and call(m=0) == 2
    assert call(gu=_mat(0)) == 2 and call(gu=_mat(128, 16416), dn=_mat(16416, 64)) == 2
    assert call(ws=None) == 1 and call(b=need - 1) == 1 and call(ws=FAKE + 128) == 3
    assert call(r=None) == 1 and call(ro=None) == 1 and call(x=None) == 1 and call(t=2) == 1
    assert call(ldr=63) == 1 and call(ldro=63) == 1 and call(ldx=63) == 1 and call(ld_gate=63) == 1
    assert call(ldro=72) == 1                                             # in place with another pitch
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1
    assert call(r=FAKE + 2) == 3 and call(ro=FAKE + 2) == 3 and call(x=FAKE + 1) == 3
    for name in ("pre_weight", "post_weight", "next_weight", "gate"):
        assert call(**{name: FAKE + 2}) == 3

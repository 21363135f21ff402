"""The C ABI of the attention sublayer and of log probabilities without a GPU:
workspace sizes, and refusals before any HIP call."""
import ctypes
import math

import pytest

from test_block_abi import FAKE, L  # noqa: F401

F32, BF16 = 0, 1


def _heads(**kw):
    from bit_fp8_codebook_amd._block import Q3HeadNorms
    d = dict(heads_q=4, heads_kv=2, head_dim=64, rotated=64, interleaved=0, eps=1e-6, q_weight=FAKE, k_weight=FAKE,
             inv_freq=FAKE)
    d.update(kw)
    return Q3HeadNorms(**d)


def _cache(**kw):
    from bit_fp8_codebook_amd._block import Q3PagedCache
    d = dict(k=FAKE, v=FAKE, pages=10, page_stride=2 * 16 * 64, page_size=16, heads=2, head_dim=64)
    d.update(kw)
    return Q3PagedCache(**d)


def _batch(**kw):
    from bit_fp8_codebook_amd._block import Q3PagedBatch
    d = dict(sequences=3, q_start=FAKE, kv_len=FAKE, page_table=FAKE, ld_table=8, table_pages=8)
    d.update(kw)
    return Q3PagedBatch(**d)


def _ref(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHES = [(dict(k=None), 1), (dict(v=None), 1), (dict(pages=0), 2), (dict(pages=1 << 32), 2), (dict(page_size=24), 2),
              (dict(page_size=0), 2), (dict(page_size=2048), 2), (dict(heads=0), 2), (dict(heads=2048), 2),
              (dict(head_dim=40), 2), (dict(head_dim=272), 2), (dict(head_dim=0), 2), (dict(page_stride=2040), 1),
              (dict(page_stride=2052), 3), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3),
              (dict(page_stride=1 << 58), 2)]
BAD_BATCHES = [(dict(sequences=0), 2), (dict(sequences=65536), 2), (dict(q_start=None), 1), (dict(kv_len=None), 1),
               (dict(page_table=None), 1), (dict(table_pages=0), 2), (dict(ld_table=7), 1), (dict(q_start=FAKE + 2), 3),
               (dict(kv_len=FAKE + 1), 3), (dict(page_table=FAKE + 2), 3)]


def test_rope_refusals(L):  # noqa: F811
    def call(h=_heads(), qkv=FAKE, ld=512, pos=FAKE, q=FAKE, ldq=256, k=FAKE, ldk=128, v=FAKE, ldv=128, cache=None,
             batch=None, m=3):
        return L.q3_qk_norm_rope(_ref(h), qkv, ld, pos, q, ldq, k, ldk, v, ldv, _ref(cache), _ref(batch), m, None)

    def paged(cache=_cache(), batch=_batch(), **kw):
        return call(k=None, v=None, cache=cache, batch=batch, **kw)
    for kw, status in ((dict(heads_q=0), 2), (dict(heads_kv=0), 2), (dict(heads_q=2048), 2), (dict(head_dim=24), 2),
                       (dict(rotated=3), 1), (dict(rotated=66), 1), (dict(rotated=-2), 1), (dict(eps=-1.0), 1),
                       (dict(eps=math.nan), 1), (dict(inv_freq=None), 1), (dict(q_weight=FAKE + 2), 3),
                       (dict(k_weight=FAKE + 1), 3), (dict(inv_freq=FAKE + 2), 3)):
        assert call(h=_heads(**kw)) == status and paged(h=_heads(**kw)) == status, kw
    for f in (call, paged):
        assert f(h=None) == 1 and f(qkv=None) == 1 and f(ld=508) == 1 and f(ld=514) == 3 and f(qkv=FAKE + 4) == 3
        assert f(m=0) == 2 and f(m=1 << 31) == 2 and f(m=-1) == 2
        assert f(q=None) == 1 and f(ldq=248) == 1 and f(ldq=260) == 3 and f(q=FAKE + 8) == 3 and f(pos=FAKE + 2) == 3
    assert call(k=None) == 1 and call(v=None) == 1 and call(ldk=120) == 1 and call(ldv=132) == 3 and call(k=FAKE + 2) == 3
    assert call(pos=None) == 1
    # rows and a cache, or half of a paged call
    assert call(cache=_cache(), batch=_batch()) == 1
    assert paged(batch=None) == 1 and paged(cache=None) == 1
    for kw, status in BAD_CACHES:
        assert paged(cache=_cache(**kw)) == status, kw
    for kw, status in BAD_BATCHES:
        assert paged(batch=_batch(**kw)) == status, kw
    assert paged(cache=_cache(heads=4, page_stride=4096)) == 2 and paged(cache=_cache(head_dim=48)) == 2


def test_rope_backward_refusals(L):  # noqa: F811
    from bit_fp8_codebook_amd._block import Q3QkvGrads
    need = L.q3_qk_norm_rope_backward_workspace_bytes
    assert need(1, 64) == 1024 * 2 * 64 * 4 and need(100000, 128) == 1024 * 2 * 128 * 4   # a row for each block
    assert need(0, 64) == 0 and need(1, 40) == 0 and need(1 << 31, 64) == 0

    def call(h=_heads(), qkv=FAKE, ld=512, pos=FAKE, m=3, ws=FAKE, b=1 << 20, null=False, **kw):
        d = dict(d_type=BF16, dq=FAKE, ld_dq=256, dk=FAKE, ld_dk=128, dv=FAKE, ld_dv=128, dqkv=FAKE, ld_dqkv=512,
                 dq_weight=FAKE, dk_weight=FAKE)
        d.update(kw)
        g = Q3QkvGrads(**d)
        return L.q3_qk_norm_rope_backward(_ref(h), qkv, ld, pos, m, None if null else ctypes.byref(g), ws, b, None)
    assert call(null=True) == 1 and call(h=None) == 1 and call(qkv=None) == 1 and call(pos=None) == 1 and call(m=0) == 2
    assert call(d_type=2) == 1 and call(dqkv=None) == 1
    assert call(h=_heads(q_weight=None)) == 1 and call(h=_heads(k_weight=None)) == 1   # a gradient without its input
    assert call(ld_dq=248) == 1 and call(ld_dk=120) == 1 and call(ld_dv=120) == 1 and call(ld_dqkv=504) == 1
    assert call(ld_dq=260) == 3 and call(dk=FAKE + 8) == 3 and call(ld_dqkv=516) == 3 and call(dqkv=FAKE + 2) == 3
    assert call(d_type=F32, ld_dq=258) == 3 and call(dq_weight=FAKE + 2) == 3 and call(dk_weight=FAKE + 1) == 3
    assert call(ws=None) == 1 and call(b=100) == 1 and call(ws=FAKE + 64) == 3 and call(pos=FAKE + 2) == 3


def test_attention_refusals(L):  # noqa: F811
    need = L.q3_paged_attention_workspace_bytes
    assert need(1, 1, 4, 2, 64) > 0
    for bad in ((0, 1, 4, 2, 64), (1 << 24, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 65536, 4, 2, 64), (1, 1, 3, 2, 64),
                (1, 1, 0, 2, 64), (1, 1, 4, 0, 64), (1, 1, 4, 2, 40), (1 << 23, 1, 512, 2, 64), (1, 65535, 256, 256, 64)):
        assert need(*bad) == 0, bad

    def call(q=FAKE, ldq=256, hq=4, cache=_cache(), batch=_batch(), scale=0.1, window=0, out=FAKE, ldo=256, lse=FAKE,
             m=3, ws=FAKE, b=1 << 40):
        return L.q3_paged_attention(q, ldq, hq, _ref(cache), _ref(batch), scale, window, out, ldo, lse, m, ws, b, None)
    assert call(cache=None) == 1 and call(batch=None) == 1
    for kw, status in BAD_CACHES:
        assert call(cache=_cache(**kw)) == status, kw
    for kw, status in BAD_BATCHES:
        assert call(batch=_batch(**kw)) == status, kw
    assert call(hq=3) == 2 and call(hq=0) == 2 and call(hq=2048, ldq=1 << 20, ldo=1 << 20) == 2
    assert call(m=0) == 2 and call(m=1 << 24) == 2 and call(m=-5) == 2
    assert call(window=-1) == 1
    for scale in (math.nan, math.inf, -math.inf, 0.0, 1e-40):
        assert call(scale=scale) == 1, scale
    assert call(q=None) == 1 and call(out=None) == 1 and call(ldq=248) == 1 and call(ldo=248) == 1
    assert call(ldq=260) == 3 and call(q=FAKE + 8) == 3 and call(ldo=260) == 3 and call(out=FAKE + 2) == 3
    assert call(lse=FAKE + 2) == 3 and call(ws=None) == 1 and call(b=16) == 1 and call(ws=FAKE + 64) == 3


def test_logprobs_refusals(L):  # noqa: F811
    need = L.q3_logprobs_workspace_bytes
    assert need(2048, 151936, 20) == 0 and need(1, 151936, 20) > need(1, 151936, 0) > 0
    assert need(0, 10, 0) == 0 and need(1, 0, 0) == 0 and need(1, (1 << 19) + 1, 0) == 0 and need(1, 10, 33) == 0
    assert need(1 << 24, 10, 0) == 0 and need(1, 10, -1) == 0

    def call(l=FAKE, m=2, n=30000, ld=30000, t=FAKE, temp=1.0, top=5, lp=FAKE, h=FAKE, ids=FAKE, tlp=FAKE, st=FAKE, ws=FAKE,
             b=1 << 30):
        return L.q3_logprobs(l, m, n, ld, t, temp, top, lp, h, ids, tlp, st, ws, b, None)
    assert call(l=None) == 1 and call(t=None) == 1 and call(lp=None) == 1
    assert call(m=0) == 2 and call(m=1 << 24) == 2 and call(n=0) == 2 and call(n=(1 << 19) + 1, ld=1 << 20) == 2
    assert call(top=33) == 2 and call(top=-1) == 2 and call(ld=29999) == 1
    for temp in (0.0, -1.0, math.nan, math.inf, 1e-39):
        assert call(temp=temp) == 1, temp
    assert call(ids=None) == 1 and call(tlp=None) == 1 and call(top=0) == 1 and call(top=0, ids=None) == 1
    assert call(l=FAKE + 2) == 3 and call(t=FAKE + 1) == 3 and call(lp=FAKE + 2) == 3 and call(h=FAKE + 2) == 3
    assert call(ids=FAKE + 2) == 3 and call(tlp=FAKE + 2) == 3 and call(st=FAKE + 8) == 3
    assert call(ws=None) == 1 and call(b=8) == 1 and call(ws=FAKE + 64) == 3

    def back(l=FAKE, m=2, n=100, ld=100, t=FAKE, temp=1.0, st=FAKE, dl=FAKE, dh=FAKE, o=FAKE + 4096, lo=100, ty=BF16):
        return L.q3_logprobs_backward(l, m, n, ld, t, temp, st, dl, dh, o, lo, ty, None)
    assert back(l=None) == 1 and back(st=None) == 1 and back(o=None) == 1 and back(t=None) == 1
    assert back(m=0) == 2 and back(n=0) == 2 and back(m=1 << 24) == 2 and back(ty=2) == 1 and back(temp=0.0) == 1
    assert back(ld=99) == 1 and back(lo=99) == 1
    assert back(o=FAKE) == 1 and back(o=FAKE, ty=F32, lo=104) == 1          # in place: the logits' type and pitch
    assert back(l=FAKE + 2) == 3 and back(st=FAKE + 8) == 3 and back(o=FAKE + 4097) == 3
    assert back(o=FAKE + 4098, ty=F32) == 3 and back(dl=FAKE + 2) == 3 and back(dh=FAKE + 2) == 3 and back(t=FAKE + 2) == 3


def test_binding_refusals():
    # Shapes, types and devices are seen before any pointer leaves the binding.
    import torch
    from bit_fp8_codebook_amd import _block as b
    bf = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    for make in (lambda: b.PagedCache(bf, bf), lambda: b.PagedCache(None, bf),
                 lambda: b.PagedBatch(torch.zeros(2), torch.zeros(1), torch.zeros(1, 4, dtype=torch.int32)),
                 lambda: b.q3_qk_norm_rope(torch.zeros(3, 512), 4, 2),
                 lambda: b.q3_qk_norm_rope_backward(torch.zeros(3, 512), 4, 2),
                 lambda: b.q3_paged_attention(torch.zeros(3, 256, dtype=torch.bfloat16), None, None),
                 lambda: b.q3_logprobs(torch.zeros(3, 10), torch.zeros(3, dtype=torch.int32)),
                 lambda: b.q3_logprobs_backward(torch.zeros(3, 10), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 4))):
        with pytest.raises(ValueError):
            make()


@pytest.mark.parametrize("name,backward", [("q3_qk_norm_rope", "q3_qk_norm_rope_backward"), ("q3_paged_attention", None),
                                           ("q3_logprobs", "q3_logprobs_backward")])
def test_autograd_is_named_at_the_call(name, backward):
    from bit_fp8_codebook_amd import _block
    said = " ".join(getattr(_block, name).__doc__.split())
    assert "recorded by autograd" in said
    assert not backward or (backward in said and callable(getattr(_block, backward)))

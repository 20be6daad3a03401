"""Refusals of the linear- and softmax-attention entry points, on the host: these calls return
before any CUDA work, so they run without a GPU."""

import pytest

P = 1 << 20


@pytest.fixture(scope="module")
def g():
    import gated_delta_rule_79_b200 as pkg
    return pkg


def test_lin_prefill_refuses(g):
    def call(**kw):
        a = dict(q=P, k=P, v=P, decay=P, s0=None, o=P, sf=None, B=1, T=8, H=2, dk=64, dv=128, t=1,
                 ws=P, nws=1 << 30)
        a.update(kw)
        return g.lib.lin_prefill(*a.values(), None)
    assert call(dk=48) == g.GDR_ERR_UNSUPPORTED
    assert "d_k=48" in g.lib.gdr_last_error().decode()
    assert call(dv=256) == g.GDR_ERR_UNSUPPORTED
    assert call(T=-1) == g.GDR_ERR_INVALID_ARG
    assert call(t=2) == g.GDR_ERR_INVALID_ARG
    assert call(q=None) == g.GDR_ERR_INVALID_ARG
    assert call(k=P + 8) == g.GDR_ERR_INVALID_ARG
    assert call(decay=P + 2) == g.GDR_ERR_INVALID_ARG
    assert call(sf=P + 4) == g.GDR_ERR_INVALID_ARG
    assert call(ws=None) == g.GDR_ERR_INVALID_ARG
    assert call(nws=16) == g.GDR_ERR_INVALID_ARG
    assert call(ws=P + 16) == g.GDR_ERR_INVALID_ARG
    assert call(T=1 << 29) == g.GDR_ERR_INVALID_ARG
    assert call(B=0) == g.GDR_OK and call(H=0) == g.GDR_OK
    assert call(T=0, q=None, ws=None) == g.GDR_OK
    assert g.lib.gdr_last_error().decode() == ""


def test_lin_decode_refuses(g):
    def call(**kw):
        a = dict(q=P, k=P, v=P, decay=P, state=P, o=P, N=2, H=2, dk=64, dv=64, t=1)
        a.update(kw)
        return g.lib.lin_decode(*a.values(), None)
    assert call(dk=16) == g.GDR_ERR_UNSUPPORTED
    assert call(N=-1) == g.GDR_ERR_INVALID_ARG
    assert call(state=None) == g.GDR_ERR_INVALID_ARG
    assert call(o=P + 2) == g.GDR_ERR_INVALID_ARG
    assert call(t=9) == g.GDR_ERR_INVALID_ARG
    assert call(N=0) == g.GDR_OK


def test_lin_backward_refuses(g):
    def call(**kw):
        a = dict(q=P, k=P, v=P, decay=P, s0=None, do=P, dsf=None, dq=P, dk_=P, dv_=P, ds0=P, B=1,
                 T=8, H=2, dk=64, dv=128, t=1, ws=P, nws=1 << 30)
        a.update(kw)
        return g.lib.lin_backward(*a.values(), None)
    assert call(dv=96) == g.GDR_ERR_UNSUPPORTED
    assert call(H=-1) == g.GDR_ERR_INVALID_ARG
    assert call(do=None) == g.GDR_ERR_INVALID_ARG
    assert call(ds0=None) == g.GDR_ERR_INVALID_ARG
    assert call(dq=P + 4) == g.GDR_ERR_INVALID_ARG
    assert call(nws=0) == g.GDR_ERR_INVALID_ARG
    assert call(B=0) == g.GDR_OK


def test_attn_prefill_refuses(g):
    def call(**kw):
        a = dict(q=P, k=P, v=P, lens=None, o=P, lse=None, B=1, Tq=8, Tk=16, Hq=4, Hkv=2, d=64, w=0,
                 s=0, scale=0.125, t=1, ws=P, nws=1 << 30)
        a.update(kw)
        return g.lib.attn_prefill(*a.values(), None)
    assert call(d=96) == g.GDR_ERR_UNSUPPORTED
    assert call(Hkv=3) == g.GDR_ERR_INVALID_ARG
    assert "multiple" in g.lib.gdr_last_error().decode()
    assert call(Hkv=0) == g.GDR_ERR_INVALID_ARG
    assert call(Tk=-1) == g.GDR_ERR_INVALID_ARG
    assert call(s=-1) == g.GDR_ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == g.GDR_ERR_INVALID_ARG
    assert call(t=5) == g.GDR_ERR_INVALID_ARG
    assert call(v=None) == g.GDR_ERR_INVALID_ARG
    assert call(o=P + 8) == g.GDR_ERR_INVALID_ARG
    assert call(lens=P + 2) == g.GDR_ERR_INVALID_ARG
    assert call(ws=None) == g.GDR_ERR_INVALID_ARG
    assert call(nws=255) == g.GDR_ERR_INVALID_ARG
    assert call(B=0) == g.GDR_OK and call(Tq=0) == g.GDR_OK
    assert call(Hq=0, Hkv=0) == g.GDR_OK


def test_attn_backward_refuses(g):
    def call(**kw):
        a = dict(q=P, k=P, v=P, lens=None, o=P, lse=P, do=P, dq=P, dk=P, dv=P, B=1, Tq=8, Tk=16,
                 Hq=4, Hkv=2, d=64, w=0, s=0, scale=0.125, t=1, ws=P, nws=1 << 30)
        a.update(kw)
        return g.lib.attn_backward(*a.values(), None)
    assert call(d=16) == g.GDR_ERR_UNSUPPORTED
    assert call(Hq=5) == g.GDR_ERR_INVALID_ARG
    assert call(lse=None) == g.GDR_ERR_INVALID_ARG
    assert call(dk=None) == g.GDR_ERR_INVALID_ARG
    assert call(dv=P + 4) == g.GDR_ERR_INVALID_ARG
    assert call(nws=256) == g.GDR_ERR_INVALID_ARG
    assert call(B=0) == g.GDR_OK


def test_attn_decode_refuses(g):
    def call(**kw):
        a = dict(q=P, k=None, v=None, kc=P, vc=P, table=P, lens=P, o=P, N=2, Hq=4, Hkv=2, d=64,
                 npages=8, page=16, most=4, w=0, s=0, scale=0.125, t=1, ws=P, nws=1 << 30)
        a.update(kw)
        return g.lib.attn_decode(*a.values(), None)
    assert call(page=24) == g.GDR_ERR_UNSUPPORTED
    assert "page=24" in g.lib.gdr_last_error().decode()
    assert call(page=0) == g.GDR_ERR_UNSUPPORTED
    assert call(page=8192) == g.GDR_ERR_UNSUPPORTED
    assert call(d=256) == g.GDR_ERR_UNSUPPORTED
    assert call(Hq=3) == g.GDR_ERR_INVALID_ARG
    assert call(k=P) == g.GDR_ERR_INVALID_ARG
    assert "together" in g.lib.gdr_last_error().decode()
    assert call(npages=-1) == g.GDR_ERR_INVALID_ARG
    assert call(lens=None) == g.GDR_ERR_INVALID_ARG
    assert call(table=None) == g.GDR_ERR_INVALID_ARG
    assert call(kc=P + 8) == g.GDR_ERR_INVALID_ARG
    assert call(scale=-0.5) == g.GDR_ERR_INVALID_ARG
    assert call(s=-2) == g.GDR_ERR_INVALID_ARG
    assert call(ws=None) == g.GDR_ERR_INVALID_ARG
    assert call(most=1 << 28) == g.GDR_ERR_INVALID_ARG
    assert call(N=0) == g.GDR_OK


def test_kv_append_refuses(g):
    def call(**kw):
        a = dict(k=P, v=P, kc=P, vc=P, table=P, start=P, counts=None, N=2, K=3, Hkv=2, d=64,
                 npages=8, page=16, most=4, t=1, ws=None, nws=0)
        a.update(kw)
        return g.lib.kv_append(*a.values(), None)
    assert call(page=3) == g.GDR_ERR_UNSUPPORTED
    assert call(K=-1) == g.GDR_ERR_INVALID_ARG
    assert call(start=None) == g.GDR_ERR_INVALID_ARG
    assert call(v=None) == g.GDR_ERR_INVALID_ARG
    assert call(ws=P, nws=16) == g.GDR_ERR_INVALID_ARG
    assert call(K=0) == g.GDR_OK


def test_workspace_sizes(g):
    import torch
    bf = torch.bfloat16
    assert g.lin_workspace_bytes(1, 0, 4, 64, 64, bf) >= 256
    assert g.lin_workspace_bytes(-1, 8, 4, 64, 64, bf) == 0
    assert g.lin_workspace_bytes(1, 8, 4, 60, 64, bf) == 0
    assert g.lin_workspace_bytes(1, 4096, 4, 64, 64, bf, True) >= \
        g.lin_workspace_bytes(1, 4096, 4, 64, 64, bf)
    assert g.attn_workspace_bytes(2, 100, 100, 4, 2, 64, bf) >= 256
    assert g.attn_workspace_bytes(2, 100, 100, 4, 2, 64, bf, True) >= 256 + 4 * 2 * 4 * 100
    # few queries over many keys: sums of two parts at least
    assert g.attn_workspace_bytes(1, 100, 9000, 4, 2, 64, bf) >= 256 + 2 * 4 * 100 * 66 * 4
    assert g.attn_workspace_bytes(1, 100, 9000, 4, 2, 64, bf, window=100) == 256
    assert g.attn_workspace_bytes(1, 100, 9000, 4, 2, 64, torch.float32) == 256
    assert g.attn_workspace_bytes(2, 100, 100, 4, 3, 64, bf) == 0
    assert g.attn_decode_workspace_bytes(1, 8, 1, 128, 64, 1024, bf) > 256
    assert g.attn_decode_workspace_bytes(1, 8, 1, 128, 48, 1024, bf) == 0


def test_binding_refuses_before_the_library(g):
    import torch
    x = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        g.lin_prefill(x, x, x, torch.ones(2))
    with pytest.raises(ValueError, match="CUDA"):
        g.attn_prefill(x, x, x)
    with pytest.raises(ValueError):
        g.lin_decode(x, x, x, torch.ones(2), x)

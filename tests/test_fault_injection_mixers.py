"""Failure detection of the tensor-core linear- and softmax-attention kernels without a GPU
fault: with GDR_SPIN_LIMIT=0 their first bounded wait gives up at once (what is in flight
completes and is drained), the status word says so, and the next call runs normally."""

import pytest
import torch

from _mixers import randn

pytestmark = pytest.mark.gpu


def _lin(T):
    q, k, v = (randn((1, T, 2, 128), s, "bf16").cuda() for s in (1, 2, 3))
    return q, k, v, torch.tensor([0.9, 0.99], device="cuda")


def _calls(g):
    bf = torch.bfloat16
    x = _lin(100)
    long = _lin(1500)              # several segments
    q = randn((2, 300, 4, 128), 1, "bf16").cuda()
    k, v = (randn((2, 300, 2, 128), s, "bf16").cuda() for s in (2, 3))
    kl = randn((1, 1800, 2, 128), 4, "bf16").cuda()
    lens = torch.tensor([300, 170], dtype=torch.int32, device="cuda")
    kw = dict(window=90, sinks=3, lengths=lens)
    o, lse = g.attn_prefill(q, k, v, **kw)
    return {
        "lin_prefill": (lambda ws: g.lin_prefill(*x, workspace=ws)[0],
                        g.lin_workspace_bytes(1, 100, 2, 128, 128, bf)),
        "lin_prefill in segments": (lambda ws: g.lin_prefill(*long, workspace=ws)[0],
                                    g.lin_workspace_bytes(1, 1500, 2, 128, 128, bf)),
        "lin_backward": (lambda ws: g.lin_backward(*long, None, long[2], workspace=ws)[0],
                         g.lin_workspace_bytes(1, 1500, 2, 128, 128, bf, True)),
        "attn_prefill": (lambda ws: g.attn_prefill(q, k, v, workspace=ws, **kw)[0],
                         g.attn_workspace_bytes(2, 300, 300, 4, 2, 128, bf)),
        "attn_prefill in parts": (lambda ws: g.attn_prefill(kl[:, :90], kl, kl, workspace=ws)[0],
                                  g.attn_workspace_bytes(1, 90, 1800, 2, 2, 128, bf)),
        "attn_backward": (lambda ws: g.attn_backward(q, k, v, o, lse, q, workspace=ws, **kw)[1],
                          g.attn_workspace_bytes(2, 300, 300, 4, 2, 128, bf, True, 90, 3)),
    }


@pytest.mark.parametrize("name", ["lin_prefill", "lin_prefill in segments", "lin_backward",
                                  "attn_prefill", "attn_prefill in parts", "attn_backward"])
def test_bounded_waits_report_and_recover(name, monkeypatch):
    import gated_delta_rule_79_b200 as g
    call, size = _calls(g)[name]
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    good = call(ws)
    g.workspace_status(ws)
    monkeypatch.setenv("GDR_SPIN_LIMIT", "0")
    call(ws)
    with pytest.raises(g.GdrError) as e:
        g.workspace_status(ws)
    assert e.value.status == g.GDR_ERR_TIMEOUT
    monkeypatch.delenv("GDR_SPIN_LIMIT")
    again = call(ws)
    g.workspace_status(ws)
    assert torch.equal(good, again)

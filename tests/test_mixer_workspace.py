"""The status of linear- and softmax-attention calls that are given no workspace: what a kernel
records stays readable through mixer_workspace(), a stream at a time."""

import threading

import pytest
import torch

from _mixers import randn

pytestmark = pytest.mark.gpu


def _decode(g, pages, n, **kw):
    """A step of one sequence of n tokens over the given page table."""
    q = randn((1, 4, 64), 1, "bf16").cuda()
    kc, vc = randn((4, 16, 2, 64), 2, "bf16").cuda(), randn((4, 16, 2, 64), 3, "bf16").cuda()
    t = torch.tensor([pages], dtype=torch.int32, device="cuda")
    return g.attn_decode(q, kc, vc, t, torch.tensor([n], dtype=torch.int32, device="cuda"), **kw)


def _status(g, **kw):
    """0, or the status that the kept workspace holds."""
    try:
        g.workspace_status(g.mixer_workspace(**kw), **kw)
    except g.GdrError as e:
        return e.status
    return 0


def test_bad_pages_and_positions_are_on_record():
    import gated_delta_rule_79_b200 as g
    _status(g)
    _decode(g, [0, 1], 20)
    assert _status(g) == 0
    _decode(g, [0, 7], 20)
    _decode(g, [0, 1], 20)                   # good calls leave the record alone
    assert _status(g) == g.GDR_ERR_INVALID_ARG and _status(g) == 0
    k = randn((1, 1, 2, 64), 2, "bf16").cuda()
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.tensor([[0]], dtype=torch.int32, device="cuda")
    g.kv_append(k, k, cache, cache.clone(), one, torch.tensor([16], dtype=torch.int32, device="cuda"))
    assert _status(g) == g.GDR_ERR_INVALID_ARG


def test_waits_that_gave_up_are_on_record(monkeypatch):
    """(GDR_SPIN_LIMIT=0: every bounded wait gives up at once, and what is in flight is drained.)"""
    import gated_delta_rule_79_b200 as g
    _status(g)
    x = [randn((1, 200, 2, 64), s, "bf16").cuda() for s in (1, 2, 3)]
    decay = torch.tensor([0.9, 0.99], device="cuda")
    o, lse = g.attn_prefill(*x)
    calls = (lambda: g.attn_prefill(*x), lambda: g.attn_backward(*x, o, lse, x[0]),
             lambda: g.lin_prefill(*x, decay), lambda: g.lin_backward(*x, decay, None, x[2]))
    for call in calls:
        good = call()
        assert _status(g) == 0
        monkeypatch.setenv("GDR_SPIN_LIMIT", "0")
        call()
        monkeypatch.delenv("GDR_SPIN_LIMIT")
        assert _status(g) == g.GDR_ERR_TIMEOUT
        assert all(torch.equal(a, b) for a, b in zip(good, call())) and _status(g) == 0


def test_each_stream_has_its_own_and_a_larger_call_keeps_the_record():
    import gated_delta_rule_79_b200 as g
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _status(g), _status(g, stream=side)
    _decode(g, [0, 7], 20, stream=side)
    assert _status(g) == 0
    before = g.mixer_workspace(stream=side)
    with torch.cuda.stream(side):
        q, k = (randn((1, t, 4, 64), 1, "bf16").cuda() for t in (300, 9000))
        g.attn_prefill(q, k, k)              # parts: more workspace than there is
    after = g.mixer_workspace(stream=side)
    assert after.numel() > before.numel()
    assert _status(g, stream=side) == g.GDR_ERR_INVALID_ARG and _status(g) == 0


def test_a_given_workspace_and_a_captured_call_do_not_touch_it():
    import gated_delta_rule_79_b200 as g
    _status(g)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    _decode(g, [0, 7], 20, workspace=ws)
    assert _status(g) == 0
    kept = g.mixer_workspace().clone()
    q, k = (randn((1, t, 4, 64), 1, "bf16").cuda() for t in (300, 9000))
    ref = g.attn_prefill(q, k, k)[0]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = g.attn_prefill(q, k, k)[0]
        graphs.append((graph, out))
    first = g.mixer_workspace()
    big = randn((2, 600, 4, 64), 2, "bf16").cuda(), randn((2, 20000, 4, 64), 3, "bf16").cuda()
    g.attn_prefill(big[0], big[1], big[1])          # the kept workspace may be another one now
    del first, kept
    for graph, out in graphs:
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_threads_on_one_stream():
    """Calls of several threads that share a stream and its workspace, each of several kernels."""
    import gated_delta_rule_79_b200 as g
    xs = []
    for s in range(4):
        q, k, v = (randn((1, t, 4, 64), s + 10 * i, "bf16").cuda()
                   for i, t in enumerate((300, 6000, 6000)))
        xs.append((q, k, v, g.attn_prefill(q, k, v)[0]))
    torch.cuda.synchronize()
    bad = []

    def work(q, k, v, ref):
        outs = [g.attn_prefill(q, k, v)[0] for _ in range(200)]
        torch.cuda.synchronize()
        bad.extend(i for i, o in enumerate(outs) if not torch.equal(o, ref))
    ts = [threading.Thread(target=work, args=x) for x in xs]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad

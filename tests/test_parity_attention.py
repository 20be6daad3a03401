"""Sliding-window attention (attn_prefill, attn_backward) against the fp64 oracle, element by
element within counted roundings (_mixers.py)."""

import numpy as np
import pytest
import torch

from oracle import attention, attention_backward
from _mixers import BF16, DT, F32, close, randn, to64, unit

pytestmark = pytest.mark.gpu


def _inputs(B, Tq, Tk, Hq, Hkv, d, dtype, seed=0):
    return (randn((B, Tq, Hq, d), seed, dtype), randn((B, Tk, Hkv, d), seed + 1, dtype),
            randn((B, Tk, Hkv, d), seed + 2, dtype))


def _lens(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def _forward(q, k, v, dtype, lengths=None, **kw):
    import gated_delta_rule_79_b200 as g
    o, lse = g.attn_prefill(q.cuda(), k.cuda(), v.cuda(), lengths=_lens(lengths), **kw)
    torch.cuda.synchronize()
    assert o.dtype == DT[dtype] and lse.dtype == torch.float32
    ref, lse_ref, mag = attention(to64(q), to64(k), to64(v), lengths=lengths, magnitude=True, **kw)
    u = unit(dtype)
    bound = u * np.abs(ref) * (1 + 2 * u) + u * mag + F32 * 4 * mag + 1e-30
    close(to64(o), ref, bound, "o")
    close(to64(lse), lse_ref, F32 * (1 + np.abs(np.where(np.isfinite(lse_ref), lse_ref, 0))), "lse")
    return o, lse


def _check(q, k, v, dtype, lengths=None, seed=7, **kw):
    import gated_delta_rule_79_b200 as g
    o, lse = _forward(q, k, v, dtype, lengths, **kw)
    do = randn(q.shape, seed, dtype)
    got = g.attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), lengths=_lens(lengths), **kw)
    torch.cuda.synchronize()
    # fp32: every exponent is a product of two rounded factors near 10, F32 covers it
    u = unit(dtype)
    ref, rounding = attention_backward(to64(q), to64(k), to64(v), to64(do), lengths=lengths,
                                       unit=u + F32, **kw)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, rounding):
        assert x.dtype == DT[dtype]
        close(to64(x), r, u * np.abs(r) * (1 + 2 * u) + 1.02 * b + 1e-30, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 129, 300])
def test_causal(dtype, d, T):
    _check(*_inputs(2, T, T, 2, 2, d, dtype, T), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 0), (64, 4), (100, 1), (130, 70),
                                          (128, 200), (299, 2), (10 ** 9, 5)])
def test_windows_and_sinks(dtype, d, window, sinks):
    _check(*_inputs(1, 300, 300, 2, 1, d, dtype, 3), dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (8, 1), (5, 5)])
def test_grouped_heads(dtype, Hq, Hkv):
    _check(*_inputs(2, 150, 150, Hq, Hkv, 128, dtype, 11), dtype, window=90, sinks=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks,lengths", [(100, 3, None), (0, 0, None), (50, 140, [2100])])
def test_keys_that_many_queries_see(dtype, window, sinks, lengths):
    """Key tiles with sinks, and early ones without a window, are cut along their queries."""
    _check(*_inputs(1, 2600, 2600, 4, 1, 64, dtype, 5), dtype, lengths, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(1, 400), (5, 131), (130, 513), (200, 70), (3, 1)])
def test_part_of_a_prompt(dtype, Tq, Tk):
    """The last Tq positions of Tk; with more queries than keys the first ones see nothing."""
    _check(*_inputs(2, Tq, Tk, 4, 2, 64, dtype, Tq), dtype)
    _check(*_inputs(1, Tq, Tk, 4, 2, 128, dtype, Tq), dtype, window=33, sinks=4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_padded_batch_with_anything_behind_the_lengths(dtype, d):
    B, T = 5, 270
    q, k, v = _inputs(B, T, T, 4, 2, d, dtype, 2)
    lens = [270, 0, 1, 128, 201]
    for x in (q, k, v):
        for b, n in enumerate(lens):
            x[b, n:] = float("nan")
    _check_padded(q, k, v, dtype, lens, window=0)
    _check_padded(q, k, v, dtype, lens, window=50, sinks=3)


def _check_padded(q, k, v, dtype, lens, **kw):
    import gated_delta_rule_79_b200 as g
    o, lse = _forward(q, k, v, dtype, lens, **kw)
    do = randn(q.shape, 5, dtype)
    for b, n in enumerate(lens):
        do[b, max(0, n - (k.shape[1] - q.shape[1])):] = float("inf")
    got = g.attn_backward(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), lengths=_lens(lens), **kw)
    u = unit(dtype)
    ref, rounding = attention_backward(to64(q), to64(k), to64(v), to64(do), lengths=lens, unit=u + F32, **kw)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, rounding):
        close(to64(x), r, u * np.abs(r) * (1 + 2 * u) + 1.02 * b + 1e-30, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk,lens", [(130, 300, [300, 171, 170, 169, 5, 250]), (300, 130, [130, 1, 0, 77, 64, 128])])
def test_part_of_a_padded_batch(dtype, Tq, Tk, lens):
    """Fewer queries than keys (or more) and lengths that end among them, before and after."""
    q, k, v = _inputs(6, Tq, Tk, 4, 2, 64, dtype, 9)
    for x, off in ((q, Tk - Tq), (k, 0), (v, 0)):
        for b, n in enumerate(lens):
            x[b, max(0, n - off):] = float("nan")
    _check_padded(q, k, v, dtype, lens, window=0)
    _check_padded(q, k, v, dtype, lens, window=70, sinks=5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,lens,window,sinks", [
    (1, 2000, 2, 1, None, 0, 0),                     # 15 tiles of keys for a single query
    (129, 1900, 4, 2, [1900, 1771, 1772, 0, 1, 1850], 0, 0),
    (129, 1900, 4, 2, [1900, 1771, 1772, 0, 1, 1850], 1000, 140),
    (300, 1300, 6, 2, [1300, 1290], 900, 3),         # parts of the second pair of tiles only
    (2000, 1000, 3, 1, None, 0, 0),                  # queries that see nothing, in every part
])
def test_few_queries_over_many_keys(d, Tq, Tk, Hq, Hkv, lens, window, sinks):
    """Where there are fewer query tiles than SMs their keys are cut into parts and joined."""
    q, k, v = _inputs(len(lens or [0]), Tq, Tk, Hq, Hkv, d, "bf16", 21)
    if lens is None:
        _forward(q, k, v, "bf16", window=window, sinks=sinks)
        return
    for x, off in ((q, Tk - Tq), (k, 0), (v, 0)):
        for b, n in enumerate(lens):
            x[b, max(0, n - off):] = float("nan")
    _forward(q, k, v, "bf16", lens, window=window, sinks=sinks)


def test_scores_that_lie_far_apart_in_the_parts():
    """One key far above all others, in one part: the others' weights vanish, none overflows."""
    q, k, v = _inputs(1, 40, 1800, 2, 1, 64, "bf16", 31)
    q[...] = 0.5
    k[0, 70], k[0, 1000] = 40.0, 44.0
    _forward(q, k, v, "bf16")


def test_lengths_outside_the_tensor_are_clamped():
    import gated_delta_rule_79_b200 as g
    q, k, v = (x.cuda() for x in _inputs(2, 70, 70, 2, 2, 64, "bf16"))
    o, lse = g.attn_prefill(q, k, v, lengths=_lens([10 ** 6, -3]))
    full, lse_full = g.attn_prefill(q, k, v)
    assert torch.equal(o[0], full[0]) and torch.equal(lse[0], lse_full[0])
    assert torch.count_nonzero(o[1]) == 0 and (lse[1] == -np.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores_and_scale(dtype):
    """Scores in the hundreds, rising along the keys, so that the running maximum moves."""
    q, k, v = _inputs(1, 260, 260, 2, 2, 64, dtype, 4)
    ramp = torch.linspace(0.5, 20, 260).view(1, -1, 1, 1)
    q, k = (q * 4).to(q.dtype), (k * ramp).to(k.dtype)
    import gated_delta_rule_79_b200 as g
    o, lse = g.attn_prefill(q.cuda(), k.cuda(), v.cuda(), scale=0.3)
    ref, lse_ref, mag = attention(to64(q), to64(k), to64(v), scale=0.3, magnitude=True)
    # an exponent of magnitude E carries E roundings of fp32 (each 2^-24) into every weight
    e = 0.3 * np.einsum("bihd,bjhd->bhij", np.abs(to64(q)), np.abs(to64(k))).max() * 2.0 ** -22
    u = unit(dtype)
    close(to64(o), ref, u * np.abs(ref) * (1 + 2 * u) + (u + F32 * 4 + 2 * e) * mag, "o")
    close(to64(lse), lse_ref, F32 * (1 + np.abs(lse_ref)) + e, "lse")


def test_no_keys_and_no_queries():
    import gated_delta_rule_79_b200 as g
    q = torch.ones(2, 3, 4, 64, device="cuda", dtype=torch.bfloat16)
    k = torch.ones(2, 0, 2, 64, device="cuda", dtype=torch.bfloat16)
    o, lse = g.attn_prefill(q, k, k)
    assert torch.count_nonzero(o) == 0 and (lse == -np.inf).all()
    dq, dk, dv = g.attn_backward(q, k, k, o, lse, q)
    assert torch.count_nonzero(dq) == 0 and dk.shape == k.shape
    o, lse = g.attn_prefill(k.new_ones(2, 0, 2, 64), q[:, :, :2].contiguous(), q[:, :, :2].contiguous())
    assert o.shape == (2, 0, 2, 64)
    x = q[:, :, :2].contiguous()
    dq, dk, dv = g.attn_backward(o, x, x, o, lse, o)
    assert torch.count_nonzero(dk) == 0 and torch.count_nonzero(dv) == 0


def test_without_lse_and_given_outputs():
    import gated_delta_rule_79_b200 as g
    q, k, v = (x.cuda() for x in _inputs(1, 200, 200, 2, 2, 128, "bf16"))
    o, lse = g.attn_prefill(q, k, v, window=40)
    o2, none = g.attn_prefill(q, k, v, window=40, lse=False, o=torch.full_like(o, 7))
    assert none is None and torch.equal(o, o2)


def test_backward_by_differences():
    """Along one direction of each input, in fp32: central differences of the forward kernel."""
    import gated_delta_rule_79_b200 as g
    q, k, v = (x.cuda() for x in _inputs(1, 90, 90, 4, 2, 64, "f32", 8))
    kw = dict(window=30, sinks=2)
    do = randn(q.shape, 3).cuda()

    def loss(*x):
        return (g.attn_prefill(*x, **kw)[0].double() * do).sum().item()
    o, lse = g.attn_prefill(q, k, v, **kw)
    grads = g.attn_backward(q, k, v, o, lse, do, **kw)
    h = 2.0 ** -7
    for i, gr in enumerate(grads):
        e = randn(gr.shape, 30 + i).cuda()
        up, down = [q, k, v], [q, k, v]
        up[i], down[i] = up[i] + h * e, down[i] - h * e
        slope = (loss(*up) - loss(*down)) / (2 * h)
        want = (gr.double() * e).sum().item()
        # third derivatives times h^2 / 6, and fp32 sums divided by h
        assert abs(slope - want) <= 2e-3 * (gr.double() * e).norm().item() * gr.numel() ** 0.5 ** 0.5 + 1e-2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_deterministic_streams_and_graphs(dtype):
    import gated_delta_rule_79_b200 as g
    q, k, v = (x.cuda() for x in _inputs(2, 333, 333, 4, 2, 128, dtype))
    do = randn(q.shape, 3, dtype).cuda()
    kw = dict(window=100, sinks=3)
    o, lse = g.attn_prefill(q, k, v, **kw)
    ref = [o, lse, *g.attn_backward(q, k, v, o, lse, do, **kw)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = [*g.attn_prefill(q, k, v, stream=side, **kw)]
    a += g.attn_backward(q, k, v, *a, do, stream=side, **kw)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = [*g.attn_prefill(q, k, v, **kw)]
        b += g.attn_backward(q, k, v, *b, do, **kw)
    for x in b:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(ref, a, b):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_long_prompt_sampled():
    """A window of 4096 over 9000 tokens (bf16): sampled rows against 64 bits."""
    import gated_delta_rule_79_b200 as g
    T, W, S = 9000, 4096, 4
    q, k, v = (x.cuda() for x in _inputs(1, T, T, 4, 1, 128, "bf16", 6))
    o, lse = g.attn_prefill(q, k, v, window=W, sinks=S)
    kk, vv = k[0, :, 0].double(), v[0, :, 0].double()
    for i in (0, 1, 127, 128, 4095, 4096, 4097, 4100, 4223, 5000, 8191, 8999):
        keep = torch.zeros(T, dtype=torch.bool, device="cuda")
        keep[max(0, i - W + 1):i + 1] = True
        keep[:min(S, i + 1)] = True
        s = (q[0, i].double() @ kk.T) / 128 ** 0.5
        s[:, ~keep] = -float("inf")
        p = torch.softmax(s, -1)
        ref, mag = p @ vv, p @ vv.abs()
        close(to64(o[0, i]), to64(ref), BF16 * 1.01 * (np.abs(to64(ref)) + to64(mag)) + F32, f"row {i}")
        close(to64(lse[0, :, i]), to64(torch.logsumexp(s, -1)), F32 * 12, f"lse {i}")

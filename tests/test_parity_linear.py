"""Linear attention with one decay per head (lin_prefill, lin_decode, lin_backward) against
the fp64 oracle, element by element within counted roundings (_mixers.py)."""

import numpy as np
import pytest
import torch

from oracle import linear_attention, linear_attention_backward
from _mixers import DT, F32, close, lin_magnitude, out_bound, randn, to64

pytestmark = pytest.mark.gpu

SIZES = [(32, 32), (64, 64), (128, 128), (64, 128), (128, 64), (32, 128)]


def _inputs(B, T, H, dk, dv, dtype, state=True, seed=0):
    q = randn((B, T, H, dk), seed, dtype, dk ** -0.5)
    k, v = randn((B, T, H, dk), seed + 1, dtype), randn((B, T, H, dv), seed + 2, dtype)
    # memories from none to everything
    decay = torch.tensor([0.97, 0.5, 1.0, 0.0, 0.999, 1e-3])[torch.arange(H) % 6].contiguous()
    s0 = randn((B, H, dv, dk), seed + 3) if state else None
    return q, k, v, decay, s0


def _cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


def _check_prefill(x, dtype, label="", **kw):
    import gated_delta_rule_79_b200 as g
    o, s = g.lin_prefill(*_cuda(*x), **kw)
    torch.cuda.synchronize()
    assert o.dtype == DT[dtype]
    q, k, v, a, s0 = [to64(t) for t in x]
    o_ref, s_ref = linear_attention(q, k, v, a, s0)
    mag, fine, tot = lin_magnitude(q, k, v, a, s0)
    close(to64(o), o_ref, out_bound(o_ref, mag, fine, dtype), label + " o")
    close(to64(s), s_ref, F32 * tot + 1e-30, label + " state")
    return o, s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("T", [1, 63, 64, 65, 200])
def test_prefill(dtype, dk, dv, T):
    _check_prefill(_inputs(2, T, 3, dk, dv, dtype, seed=T), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,H", [(1, 1030, 1), (1, 2048, 2), (3, 700, 6)])
def test_prefill_in_segments(dtype, B, T, H):
    """Few heads and many tokens: the tokens are cut into segments that run side by side."""
    _check_prefill(_inputs(B, T, H, 128, 128, dtype, seed=T), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_without_states(dtype):
    import gated_delta_rule_79_b200 as g
    x = _inputs(2, 150, 4, 128, 128, dtype, state=False)
    o, _ = _check_prefill(x, dtype)
    o2, none = g.lin_prefill(*_cuda(*x), s_final=False)
    assert none is None and torch.equal(o, o2)


def test_prefill_carries_in_place_and_in_parts():
    """Two calls that carry the state in place give what one call over all tokens gives."""
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _cuda(*_inputs(1, 300, 4, 64, 64, "f32"))
    o, s = g.lin_prefill(q, k, v, a, s0)
    S = s0.clone()
    parts = [g.lin_prefill(*(t[:, c].contiguous() for t in (q, k, v)), a, S, s_final=S)[0]
             for c in (slice(0, 131), slice(131, 300))]
    assert torch.allclose(torch.cat(parts, 1), o, atol=1e-4)
    assert torch.allclose(S, s, atol=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_segments_with_the_state_carried_in_place(dtype):
    """The last segment writes the final state over the entering one, which the first segment
    reads."""
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _cuda(*_inputs(1, 1500, 2, 128, 128, dtype))
    o, s = g.lin_prefill(q, k, v, a, s0)
    for _ in range(5):
        S = s0.clone()
        o2, _ = g.lin_prefill(q, k, v, a, S, s_final=S)
        assert torch.equal(o, o2) and torch.equal(S, s)


def test_no_tokens():
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _cuda(*_inputs(2, 0, 3, 64, 32, "bf16"))
    o, s = g.lin_prefill(q, k, v, a, s0)
    assert o.shape == (2, 0, 3, 32) and torch.equal(s, s0)
    assert torch.count_nonzero(g.lin_prefill(q, k, v, a)[1]) == 0
    out = g.lin_backward(q, k, v, a, s0, v, s0)
    assert torch.equal(out[3], s0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("N,H", [(1, 1), (3, 5), (40, 32)])
def test_decode(dtype, dk, dv, N, H):
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _inputs(N, 1, H, dk, dv, dtype, seed=N)
    S = s0.cuda()
    o = g.lin_decode(*[t[:, 0].contiguous().cuda() for t in (q, k, v)], a.cuda(), S)
    torch.cuda.synchronize()
    x = [to64(t) for t in (q, k, v, a, s0)]
    o_ref, s_ref = linear_attention(*x)
    mag, fine, tot = lin_magnitude(*x)
    close(to64(o), o_ref[:, 0], out_bound(o_ref, mag, fine, dtype)[:, 0], "o")
    close(to64(S), s_ref, F32 * tot + 1e-30, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,B,T,H", [(32, 32, 2, 70, 3), (64, 64, 1, 129, 2),
                                         (128, 128, 2, 64, 3), (128, 128, 1, 900, 2),
                                         (64, 128, 2, 333, 4), (128, 64, 1, 1, 6)])
@pytest.mark.parametrize("state", [True, False])
def test_backward(dtype, dk, dv, B, T, H, state):
    import gated_delta_rule_79_b200 as g
    x = _inputs(B, T, H, dk, dv, dtype, state, seed=5)
    do = randn((B, T, H, dv), 9, dtype)
    dsf = randn((B, H, dv, dk), 10) if state else None
    got = g.lin_backward(*_cuda(*x, do, dsf))
    torch.cuda.synchronize()
    q, k, v, a, s0 = [to64(t) for t in x]
    do, dsf = to64(do), to64(dsf)
    ref = linear_attention_backward(q, k, v, a, s0, do, dsf)

    def flip(*ts):
        return [None if t is None else np.flip(t, 1) for t in ts]

    def turn(s):
        return None if s is None else np.swapaxes(s, 2, 3)
    # the three scans the gradients are; entering a reversed one undecayed at most divides by
    # nothing, so its magnitude with the state taken one step earlier bounds it
    mq, fq_, _ = lin_magnitude(do, v, k, a, turn(s0))
    fk, fq, fv, fd = flip(k, q, v, do)
    extra = np.zeros((1, 1, 1, 1)) if dsf is None else np.abs(dsf)
    mv, fv_, tot = lin_magnitude(fk, fq, fd, a, dsf, first=T % 64 or 64)
    mk, fk_, _ = lin_magnitude(fv, fd, fq, a, turn(dsf), first=T % 64 or 64)
    if dsf is not None:       # the first chunk's tokens meet it with a^i, not a^(i+1)
        for i in range(min(T, T % 64 or 64)):
            w = np.asarray(a) ** i
            more = np.einsum("h,bhvk,bhk->bhv", w, extra, np.abs(fk[:, i]))
            mv[:, i] += more
            fv_[:, i] += more
            more = np.einsum("h,bhvk,bhv->bhk", w, extra, np.abs(fv[:, i]))
            mk[:, i] += more
            fk_[:, i] += more
    close(to64(got[0]), ref[0], out_bound(ref[0], mq, fq_, dtype), "dq")
    close(to64(got[1]), ref[1], out_bound(ref[1], np.flip(mk, 1), np.flip(fk_, 1), dtype), "dk")
    close(to64(got[2]), ref[2], out_bound(ref[2], np.flip(mv, 1), np.flip(fv_, 1), dtype), "dv")
    close(to64(got[3]), ref[3], F32 * tot + 1e-30, "ds0")


def test_backward_by_differences():
    """The gradients against differences of the forward kernel itself (fp32): along one random
    direction of each input; the loss is linear in each of them alone."""
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _cuda(*_inputs(1, 150, 2, 64, 64, "f32"))
    do, dsf = randn(v.shape, 4).cuda(), randn(s0.shape, 5).cuda()

    def loss(q, k, v, s0):
        o, s = g.lin_prefill(q, k, v, a, s0)
        return ((o.double() * do).sum() + (s.double() * dsf).sum()).item()
    x = [q, k, v, s0]
    grads = g.lin_backward(q, k, v, a, s0, do, dsf)
    for i, gr in enumerate(grads):
        e = randn(x[i].shape, 20 + i).cuda()
        up, down = [y for y in x], [y for y in x]
        up[i], down[i] = x[i] + e, x[i] - e
        slope = (loss(*up) - loss(*down)) / 2
        # three losses of about 1e3 each, summed from fp32 outputs: 2^-18 of their magnitudes
        scale = sum((abs(u) * abs(w)).sum().item() for u, w in ((gr, e),))
        assert abs(slope - (gr.double() * e).sum().item()) <= 2e-4 * scale


def test_deterministic_and_two_streams():
    import gated_delta_rule_79_b200 as g
    x = _cuda(*_inputs(2, 500, 4, 128, 128, "bf16"))
    do = randn(x[2].shape, 8, "bf16").cuda()
    ref, gref = g.lin_prefill(*x), g.lin_backward(*x, do, x[4])
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):
        outs.append((g.lin_prefill(*x, stream=s1), g.lin_backward(*x, do, x[4], stream=s2)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert all(torch.equal(u, w) for u, w in zip(a, ref))
        assert all(torch.equal(u, w) for u, w in zip(b, gref))


def test_captured_and_replayed():
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _cuda(*_inputs(1, 600, 2, 128, 128, "bf16"))
    do = randn(v.shape, 8, "bf16").cuda()
    g.lin_prefill(q, k, v, a, s0)
    g.lin_backward(q, k, v, a, s0, do)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, s = g.lin_prefill(q, k, v, a, s0)
        grads = g.lin_backward(q, k, v, a, s0, do)
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    o2, s2 = g.lin_prefill(q, k, v, a, s0)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    assert all(torch.equal(x, y) for x, y in zip(grads, g.lin_backward(q, k, v, a, s0, do)))


def test_prompt_then_tokens():
    """A prompt followed by single tokens from its state gives the one long prompt's outputs."""
    import gated_delta_rule_79_b200 as g
    q, k, v, a, s0 = _cuda(*_inputs(2, 140, 3, 128, 128, "f32"))
    o, s = g.lin_prefill(q, k, v, a, s0)
    _, S = g.lin_prefill(*(t[:, :130].contiguous() for t in (q, k, v)), a, s0)
    for t in range(130, 140):
        one = g.lin_decode(*(x[:, t].contiguous() for x in (q, k, v)), a, S)
        assert torch.allclose(one, o[:, t], atol=1e-4)
    assert torch.allclose(S, s, atol=1e-3)


def test_long_memory_does_not_drift():
    """A decay of 1 - 2^-14 over 60 thousand tokens: a rounding of each chunk's decay, the same
    every time, would show."""
    import gated_delta_rule_79_b200 as g
    T = 60001
    q, k, v, _, s0 = _inputs(1, T, 1, 64, 64, "f32")
    a = torch.tensor([1 - 2.0 ** -14])
    _, s = g.lin_prefill(*_cuda(q, k, v, a, s0))
    w = torch.tensor(1 - 2.0 ** -14, dtype=torch.float64) ** torch.arange(T - 1, -1, -1)
    ref = float(a[0]) ** T * s0[0, 0].double() + v[0, :, 0].double().T @ (w[:, None] * k[0, :, 0].double())
    err = (s[0, 0].double().cpu() - ref).norm() / ref.norm()
    # the state passes about T/32 fp32 steps, a random walk of 2^-24 each: sqrt(1875) * 6e-8
    assert err <= 3e-6, err

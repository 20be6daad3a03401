"""The linear- and softmax-attention oracles against closed forms and finite differences."""

import numpy as np
import pytest

from oracle import attention, attention_backward, linear_attention, linear_attention_backward

RNG = np.random.default_rng(3)


def _lin(B=2, T=7, H=2, dk=3, dv=4):
    return (RNG.standard_normal((B, T, H, dk)), RNG.standard_normal((B, T, H, dk)),
            RNG.standard_normal((B, T, H, dv)), np.array([0.9, 0.5]),
            RNG.standard_normal((B, H, dv, dk)))


def test_linear_attention_closed_form():
    q, k, v, a, s0 = _lin()
    o, S = linear_attention(q, k, v, a, s0)
    for b in range(2):
        for h in range(2):
            t = 6
            M = a[h] ** (t + 1) * s0[b, h] + sum(
                a[h] ** (t - j) * np.outer(v[b, j, h], k[b, j, h]) for j in range(t + 1))
            assert np.allclose(S[b, h], M) and np.allclose(o[b, t, h], M @ q[b, t, h])
    # decay 0: a token sees itself only
    o, S = linear_attention(q, k, v, np.zeros(2), s0)
    assert np.allclose(o, v * (q * k).sum(-1, keepdims=True))


def test_linear_attention_is_the_delta_rule_without_its_correction():
    """With keys of one token orthogonal to all before, the delta rule with beta = 1 corrects
    nothing: both mixers agree."""
    from oracle import gated_delta_rule
    T = 4
    k = np.zeros((1, T, 1, T))
    k[0, np.arange(T), 0, np.arange(T)] = 1.0
    q, v = RNG.standard_normal((1, T, 1, T)), RNG.standard_normal((1, T, 1, 3))
    o, S = linear_attention(q, k, v, np.array([0.7]))
    o2, S2 = gated_delta_rule(q, k, v, np.full((1, T, 1), 0.7), np.ones((1, T, 1)))
    assert np.allclose(o, o2) and np.allclose(S, S2)


def _differences(f, x, h=1e-6):
    g = np.empty(x.shape)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


def test_linear_gradients_by_differences():
    q, k, v, a, s0 = _lin(1, 5)
    do, dsf = RNG.standard_normal(v.shape), RNG.standard_normal(s0[:1].shape)
    s0 = s0[:1]

    def loss():
        o, S = linear_attention(q, k, v, a, s0)
        return (o * do).sum() + (S * dsf).sum()
    for got, x in zip(linear_attention_backward(q, k, v, a, s0, do, dsf), (q, k, v, s0)):
        assert np.allclose(got, _differences(loss, x), atol=1e-7)


@pytest.mark.parametrize("window,sinks,lengths", [(0, 0, None), (3, 0, None), (2, 2, [9, 4]),
                                                  (1, 1, [0, 9])])
def test_attention_rows_and_gradients(window, sinks, lengths):
    B, Tq, Tk, Hq, Hkv, d = 2, 5, 9, 4, 2, 3
    q = RNG.standard_normal((B, Tq, Hq, d))
    k, v = RNG.standard_normal((B, Tk, Hkv, d)), RNG.standard_normal((B, Tk, Hkv, d))
    do = RNG.standard_normal(q.shape)
    kw = dict(window=window, sinks=sinks, lengths=lengths)
    o, lse = attention(q, k, v, **kw)
    # one row by hand
    for b in range(B):
        n = Tk if lengths is None else lengths[b]
        for i in range(Tq):
            p = Tk - Tq + i
            js = [j for j in range(Tk) if j <= p < n and (window == 0 or p - j < window or j < sinks)]
            if not js:
                assert (o[b, i] == 0).all() and (lse[b, :, i] == -np.inf).all()
                continue
            s = np.array([q[b, i, 3] @ k[b, j, 1] for j in js]) / np.sqrt(d)
            w = np.exp(s)
            assert np.allclose(lse[b, 3, i], np.log(w.sum()))
            assert np.allclose(o[b, i, 3], sum(x * v[b, j, 1] for x, j in zip(w, js)) / w.sum())

    def loss():
        return (attention(q, k, v, **kw)[0] * do).sum()
    grads, _ = attention_backward(q, k, v, do, **kw)
    for got, x in zip(grads, (q, k, v)):
        assert np.allclose(got, _differences(loss, x), atol=1e-7)


def test_hidden_values_may_be_anything():
    q, k, v = (RNG.standard_normal((1, 4, 1, 2)) for _ in range(3))
    ref = attention(q, k, v, lengths=[2])[0]
    for x in (q, k, v):
        x[0, 2:] = np.nan
    assert np.array_equal(attention(q, k, v, lengths=[2])[0], ref)

"""Causal softmax attention with a sliding window and sinks, and its gradients, in fp64.

q, o [B, Tq, Hq, d]; k, v [B, Tk, Hkv, d]; query i at position p = Tk - Tq + i sees key j when
j <= p, j and p lie before lengths[b], and p - j < window (0: no window) or j < sinks.  Query
head h reads key head h // (Hq / Hkv).  A query that sees nothing has o = 0 and lse = -inf.
"""

import numpy as np


def visible(Tq, Tk, window=0, sinks=0, length=None):
    """[Tq, Tk] truth values of one sequence."""
    n = Tk if length is None else int(length)
    p = np.arange(Tk - Tq, Tk)[:, None]
    j = np.arange(Tk)[None, :]
    near = (p - j < window) if window > 0 else np.ones((Tq, Tk), dtype=bool)
    return (j <= p) & (j < n) & (p < n) & (near | (j < sinks))


def _weights(q, k, mask, scale):
    """Softmax weights and lse of one (batch, head)."""
    s = np.where(mask, scale * (q @ k.T), -np.inf)
    top = np.max(s, axis=1, initial=-np.inf)
    base = np.where(np.isfinite(top), top, 0.0)
    e = np.where(mask, np.exp(s - base[:, None]), 0.0)
    l = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = base + np.log(l)
    return e / np.where(l > 0, l, 1.0)[:, None], lse


def attention(q, k, v, window=0, sinks=0, scale=None, lengths=None, magnitude=False):
    """Returns (o, lse [B, Hq, Tq]); with magnitude also sum_j p_ij |v_j|, what a relative
    error of every weight can add up to."""
    B, Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, Hq, Tq), -np.inf)
    for b in range(B):
        m = visible(Tq, Tk, window, sinks, None if lengths is None else lengths[b])
        for h in range(Hq):
            # what the mask hides may hold anything
            g = h // (Hq // Hkv)
            kk, vv = _shown(k[b, :, g], m.any(0)), _shown(v[b, :, g], m.any(0))
            p, lse[b, h] = _weights(_shown(q[b, :, h], m.any(1)), kk, m, scale)
            o[b, :, h] = p @ vv
            mag[b, :, h] = p @ np.abs(vv)
    return (o, lse, mag) if magnitude else (o, lse)


def _shown(x, rows):
    return np.where(rows[:, None], x, 0.0)


def attention_backward(q, k, v, do, window=0, sinks=0, scale=None, lengths=None, unit=0.0):
    """Returns (dq, dk, dv) of L = sum <do, o>, and with them bounds on what roundings of the
    weights, of their gradients and of o by a relative `unit` each can change: (dq, dk, dv),
    (bound_q, bound_k, bound_v)."""
    B, Tq, Hq, d = q.shape
    Tk, Hkv = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    g = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    e = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    for b in range(B):
        m = visible(Tq, Tk, window, sinks, None if lengths is None else lengths[b])
        for h in range(Hq):
            c = h // (Hq // Hkv)
            kk, vv = _shown(k[b, :, c], m.any(0)), _shown(v[b, :, c], m.any(0))
            qq, dd = _shown(q[b, :, h], m.any(1)), _shown(do[b, :, h], m.any(1))
            p, _ = _weights(qq, kk, m, scale)
            o = p @ vv
            ds = scale * p * (dd @ vv.T - (dd * o).sum(1, keepdims=True))
            g[0][b, :, h] = ds @ kk
            g[1][b, :, c] += ds.T @ qq
            g[2][b, :, c] += p.T @ dd
            # o carries its own rounding and that of the weights behind it
            off = unit * (np.abs(dd) * (np.abs(o) + p @ np.abs(vv))).sum(1, keepdims=True)
            eds = unit * np.abs(ds) + scale * p * off
            e[0][b, :, h] = eds @ np.abs(kk)
            e[1][b, :, c] += eds.T @ np.abs(qq)
            e[2][b, :, c] += unit * (p.T @ np.abs(dd))
    return tuple(g), tuple(e)

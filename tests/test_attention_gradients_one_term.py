"""attn_backward with one-term weights (bf16, more than 512 keys a query, more than 2051 keys) for
head size 128, and for 64, against the fp64 oracle, element by element (_mixers.py)."""

import numpy as np
import pytest
import torch

from oracle import attention_backward
from _mixers import F32, close, randn, to64, unit

pytestmark = pytest.mark.gpu


def _check(Tq, Tk, Hq, Hkv, d, lens, window, sinks):
    import gated_delta_rule_79_b200 as g
    B = len(lens or [0])
    q, do = (randn((B, Tq, Hq, d), s, "bf16") for s in (1, 4))
    k, v = (randn((B, Tk, Hkv, d), s, "bf16") for s in (2, 3))
    for b, n in enumerate(lens or []):                # what lies behind a length may be anything
        for x, off in ((q, Tk - Tq), (do, Tk - Tq), (k, 0), (v, 0)):
            x[b, max(0, n - off):] = float("nan")
    kw = dict(window=window, sinks=sinks)
    t = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    qc, kc, vc, dc = (x.cuda() for x in (q, k, v, do))
    o, lse = g.attn_prefill(qc, kc, vc, lengths=t, **kw)
    got = g.attn_backward(qc, kc, vc, o, lse, dc, lengths=t, **kw)
    u = unit("bf16")
    ref, rounding = attention_backward(to64(q), to64(k), to64(v), to64(do), lengths=lens, unit=u + F32, **kw)
    for name, x, r, e in zip(("dq", "dk", "dv"), got, ref, rounding):
        x = to64(x)
        close(x, r, u * np.abs(r) * (1 + 2 * u) + 1.02 * e + 1e-30, name)
        # normwise: four roundings (the weights behind o, o inside D, p or ds, the result), independent
        # and each of an rms of 2^-8 / sqrt(3) at a mantissa of 1 and three quarters of that over all
        # mantissas: 2 x 0.75 x 2^-8 / sqrt(3), below 2^-8
        assert np.linalg.norm(x - r) <= 2.0 ** -8 * np.linalg.norm(r), name


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Tq,Tk,Hq,Hkv,lens,window,sinks", [
    (2600, 2600, 2, 1, None, 0, 0),
    (2300, 2300, 4, 2, None, 600, 5),                   # key tiles with sinks are cut into parts
    (2100, 2100, 4, 1, None, 700, 140),                 # sinks in two tiles, four heads to one
    (2200, 2200, 2, 2, [2200, 1500, 0, 1, 129], 800, 2),
    (2200, 2200, 2, 1, [1999, 640], 0, 0),
    (300, 2400, 4, 2, None, 1000, 4),                   # the last part of a prompt
    (129, 2200, 2, 1, [2200, 2072, 2071, 900], 0, 0),
    (2400, 2100, 1, 1, None, 600, 3),                   # queries that see nothing
])
def test_one_term(d, Tq, Tk, Hq, Hkv, lens, window, sinks):
    _check(Tq, Tk, Hq, Hkv, d, lens, window, sinks)

"""Inputs and bounds for the linear- and softmax-attention tests.

Bounds count roundings: rounding to a type is off by at most half a step, eps / 2 relative to
the value (bf16 2^-8, fp32 2^-24).  With bf16 tensors every kernel may round the weights that
meet the values (and the state that meets the queries) and the result, so an element may be
off by 2^-8 |result| + 2^-8 (sum of |weight| |value|); the sums themselves run in fp32, whose
own roundings stay below F32 = 2^-18 (64 half steps) of the sum of magnitudes.
"""

import numpy as np
import torch

BF16 = 2.0 ** -8
F32 = 2.0 ** -18
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def unit(dtype):
    return BF16 if dtype in ("bf16", torch.bfloat16) else 0.0


def randn(shape, seed, dtype="f32", std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(DT[dtype])


def to64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def close(x, ref, bound, label=""):
    """|x - ref| <= bound element by element (infinities equal)."""
    x, ref, bound = (np.asarray(a, dtype=np.float64) for a in (x, ref, bound))
    assert x.shape == ref.shape, (label, x.shape, ref.shape)
    inf = np.isinf(ref)
    assert np.array_equal(x[inf], ref[inf]), f"{label}: infinities differ"
    d = np.where(inf, 0.0, np.abs(np.where(inf, 0.0, x) - np.where(inf, 0.0, ref)))
    bad = ~(d <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(np.where(np.isnan(d), np.inf, d - bound))), d.shape)
        raise AssertionError(f"{label}: {int(bad.sum())} of {d.size} elements off, first at {i}: "
                             f"{x[i]:.6g} for {ref[i]:.6g}, bound {np.broadcast_to(bound, d.shape)[i]:.3g}")


def lin_magnitude(q, k, v, decay, s0, chunk=64, first=None):
    """What relative errors of the weights and of the state entering each chunk can add up to
    in o (mag), what the fp32 sums behind them add up in magnitude (fine), and the sum of
    magnitudes behind S_T.  fine takes |q|.|k| where mag takes |q.k|: a dot product of n terms
    in fp32 is off by up to n 2^-24 sum |q_c k_c|, however small the sum itself comes out.
    first: length of the first chunk.  A scan from the last token processes the chunks that
    start at multiples of 64, the ragged one first; where a chunk starts decides which tokens
    see a rounded state (error 2^-8 |S| |q|) rather than rounded weights (2^-8 |q.k| |v|)."""
    B, T, H, _ = q.shape
    mag, fine = np.zeros(v.shape), np.zeros(v.shape)
    S = np.zeros((B, H, v.shape[-1], q.shape[-1])) if s0 is None else s0.copy()
    tot = np.abs(S)
    a = np.asarray(decay, dtype=np.float64)
    first = min(first or chunk, T)
    for c in [0, *range(first, T, chunk)] if T else []:
        L = first if c == 0 else min(chunk, T - c)
        i = np.arange(L)
        for b in range(B):
            for h in range(H):
                qq, kk, vv = q[b, c:c + L, h], k[b, c:c + L, h], v[b, c:c + L, h]
                D = np.tril(a[h] ** np.maximum(i[:, None] - i[None, :], 0))
                mag[b, c:c + L, h] = (np.abs(qq @ kk.T) * D) @ np.abs(vv) + \
                    (a[h] ** (i + 1))[:, None] * (np.abs(qq) @ np.abs(S[b, h]).T)
                fine[b, c:c + L, h] = (np.abs(qq) @ np.abs(kk).T * D) @ np.abs(vv) + \
                    (a[h] ** (i + 1))[:, None] * (np.abs(qq) @ tot[b, h].T)
                w = (a[h] ** (L - 1 - i))[:, None] * kk
                S[b, h] = a[h] ** L * S[b, h] + vv.T @ w
                tot[b, h] = a[h] ** L * tot[b, h] + np.abs(vv).T @ np.abs(w)
    return mag, fine, tot


def out_bound(ref, mag, fine, dtype):
    u = unit(dtype)
    # two of the rounded operands, the result, and the fp32 sums
    return u * np.abs(ref) * (1 + 2 * u) + 2 * u * mag + F32 * fine + 1e-30

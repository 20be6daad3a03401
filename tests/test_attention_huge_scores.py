"""Finite queries and keys whose scores are so large that the rounding of one score passes 100:
every weight is then 0 or shared by equal scores, and o is finite.

Queries and keys are powers of two times small whole numbers, so that every q.k is exact in fp32
and equal scores are equal; scores that differ, differ by more than 2^24."""

import numpy as np
import pytest
import torch

from oracle import attention
from _mixers import DT, F32, close, randn, to64, unit

pytestmark = pytest.mark.gpu


def _inputs(Tq, Tk, Hq, Hkv, d, dtype, sign, power):
    g = torch.Generator().manual_seed(Tk + d)
    n = torch.randint(1, 8, (1, Tk, Hkv, 1), generator=g)
    n[0, Tk // 2:, :, 0] += 1                      # (so that the maximum moves along the keys)
    q = torch.full((1, Tq, Hq, d), 2.0 ** power).to(DT[dtype])
    k = (sign * 2.0 ** power * n.float()).expand(1, Tk, Hkv, d).to(DT[dtype]).contiguous()
    return q, k, randn((1, Tk, Hkv, d), 3, dtype)


def _compare(o, q, k, v, dtype, label, **kw):
    ref, lse, mag = attention(to64(q), to64(k), to64(v), magnitude=True, **kw)
    u = unit(dtype)
    assert torch.isfinite(o).all(), label
    close(to64(o), ref, u * np.abs(ref) * (1 + 2 * u) + (u + 4 * F32) * mag + 1e-30, label)
    return lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [13, 15, 25, 50])
@pytest.mark.parametrize("Tq,Tk,window,sinks", [(300, 300, 0, 0), (300, 300, 70, 3), (40, 1800, 0, 0)])
def test_prefill(dtype, d, sign, power, Tq, Tk, window, sinks):
    import gated_delta_rule_79_b200 as g
    q, k, v = _inputs(Tq, Tk, 2, 1, d, dtype, sign, power)
    for scale in (None, 0.3):
        o, lse = g.attn_prefill(q.cuda(), k.cuda(), v.cuda(), window=window, sinks=sinks, scale=scale)
        ref = _compare(o, q, k, v, dtype, f"o, scale {scale}", window=window, sinks=sinks, scale=scale)
        close(to64(lse), ref, F32 * (1 + np.abs(ref)), "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [15, 50])
def test_decode(dtype, d, sign, power):
    import gated_delta_rule_79_b200 as g
    q, k, v = _inputs(1, 800, 4, 2, d, dtype, sign, power)
    table = torch.arange(50, dtype=torch.int32, device="cuda")[None]
    o = g.attn_decode(q[:, 0].cuda().contiguous(), k.view(50, 16, 2, d).cuda(), v.view(50, 16, 2, d).cuda(),
                      table, torch.tensor([800], dtype=torch.int32, device="cuda"), scale=0.3)
    _compare(o[None], q, k, v, dtype, "o", scale=0.3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Tq,Tk", [(300, 900), (40, 1800)])
def test_small_differences_of_large_scores(d, Tq, Tk):
    """Scores of 2^20 (exact in fp32) that rise by some units along the keys, so that weights of the
    tiles before count still: what was summed is carried over between the rounded bases."""
    import gated_delta_rule_79_b200 as g
    gen = torch.Generator().manual_seed(d)
    q = torch.zeros(1, Tq, 2, d)
    k = torch.zeros(1, Tk, 1, d)
    q[..., 0], k[..., 0] = 2.0 ** 10, 2.0 ** 10
    # whole numbers of eighths, 12 more from one tile of 128 keys to the next
    q[..., 1], q[..., 2] = 1.0, 1.0
    k[..., 1] = torch.randint(-8, 9, (1, Tk, 1), generator=gen) / 8
    k[..., 2] = (torch.arange(Tk) // 128 * 12).view(1, Tk, 1)
    q, k, v = q.bfloat16(), k.bfloat16(), randn((1, Tk, 1, d), 5, "bf16")
    o, lse = g.attn_prefill(q.cuda(), k.cuda(), v.cuda(), scale=0.7)
    ref = _compare(o, q, k, v, "bf16", "o", scale=0.7)
    close(to64(lse), ref, F32 * (1 + np.abs(ref)), "lse")

"""Queries over no keys at all (Tk = 0): o = 0 and lse = -inf, in given outputs too."""

import pytest
import torch

from _mixers import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,Tq,Hq,Hkv", [(1, 1, 1, 1), (3, 85, 3, 1), (2, 300, 4, 2)])
def test_no_keys(dtype, d, B, Tq, Hq, Hkv):
    import gated_delta_rule_79_b200 as g
    q = torch.full((B, Tq, Hq, d), float("nan"), dtype=DT[dtype], device="cuda")
    k = torch.empty(B, 0, Hkv, d, dtype=DT[dtype], device="cuda")
    # an element more on either side stays as it is
    lse = torch.full((B * Hq * Tq + 8,), 7.0, device="cuda")
    o = torch.full((B * Tq * Hq * d + 16,), 7.0, dtype=DT[dtype], device="cuda")
    got, got_lse = g.attn_prefill(q, k, k, window=5, sinks=1, o=o[8:-8].view(q.shape),
                                  lse=lse[4:-4].view(B, Hq, Tq))
    assert torch.count_nonzero(got) == 0 and (got_lse == -float("inf")).all()
    assert (o[:8] == 7).all() and (o[-8:] == 7).all() and (lse[:4] == 7).all() and (lse[-4:] == 7).all()
    o2, none = g.attn_prefill(q, k, k, lse=False, lengths=torch.zeros(B, dtype=torch.int32, device="cuda"))
    assert none is None and torch.count_nonzero(o2) == 0

"""attn_decode's new token where its own page lies outside the pool: it is neither stored nor
seen, like every other token of such a page, and the status word says so."""

import numpy as np
import pytest
import torch

from oracle import attention
from _mixers import DT, F32, close, randn, to64, unit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_new_token_on_a_page_outside_the_pool_is_left_out(dtype, d, window, sinks):
    import gated_delta_rule_79_b200 as g
    N, Hq, Hkv, page, per = 4, 4, 2, 16, 6
    # the new token: first of its page, in the middle of it, the sequence's only one, and a good one
    lens = [65, 73, 1, 40]
    table = torch.randperm(N * per, generator=torch.Generator().manual_seed(1)).view(N, per).int()
    bad = table.clone()
    bad[0, 4], bad[1, 4], bad[2, 0] = N * per, -1, 2 ** 31 - 1
    kc = randn((N * per, page, Hkv, d), 1, dtype).cuda()
    vc = randn((N * per, page, Hkv, d), 2, dtype).cuda()
    q, k, v = randn((N, Hq, d), 3, dtype), randn((N, Hkv, d), 4, dtype), randn((N, Hkv, d), 5, dtype)
    before = kc.clone(), vc.clone()
    ws = torch.zeros(g.attn_decode_workspace_bytes(N, Hq, Hkv, d, page, per, DT[dtype], window, sinks),
                     dtype=torch.uint8, device="cuda")
    o = g.attn_decode(q.cuda(), kc, vc, bad.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                      k=k.cuda(), v=v.cuda(), window=window, sinks=sinks, workspace=ws)
    with pytest.raises(g.GdrError) as e:
        g.workspace_status(ws)
    assert e.value.status == g.GDR_ERR_INVALID_ARG
    # only the good sequence's token was stored
    before[0][table[3, 2].long(), 39 % page], before[1][table[3, 2].long(), 39 % page] = k[3].cuda(), v[3].cuda()
    assert torch.equal(kc, before[0]) and torch.equal(vc, before[1])
    u = unit(dtype)
    for n, length in enumerate(lens):
        # the tokens that the mask shows and whose pages are in the pool
        t = [j for j in range(length)
             if (not window or length - 1 - j < window or j < sinks)
             and 0 <= int(bad[n, j // page]) < N * per]
        if not t:
            assert torch.count_nonzero(o[n]) == 0
            continue
        at = table[n].long()[torch.tensor(t) // page], torch.tensor(t) % page
        ref, _, mag = attention(to64(q[n])[None, None], to64(kc.cpu()[at])[None], to64(vc.cpu()[at])[None],
                                magnitude=True)
        close(to64(o[n]), ref[0, 0], u * np.abs(ref[0, 0]) * (1 + 2 * u) + (u + 4 * F32) * mag[0, 0] + 1e-30,
              f"sequence {n}")

"""One-token attention over a paged cache (attn_decode, kv_append) against the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import attention
from _mixers import DT, F32, close, randn, to64, unit

pytestmark = pytest.mark.gpu


class Cache:
    """Sequences of given lengths in shuffled pages; what no sequence holds is NaN."""

    def __init__(self, lens, Hkv, d, page, dtype, extra=2, seed=0):
        N, most = len(lens), max([1, *lens])
        self.per = -(-most // page) + extra
        npages = N * self.per + 3
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(npages, generator=g)[:N * self.per].view(N, self.per).int()
        self.k = [randn((n, Hkv, d), seed + 10 * i + 1, dtype) for i, n in enumerate(lens)]
        self.v = [randn((n, Hkv, d), seed + 10 * i + 2, dtype) for i, n in enumerate(lens)]
        shape = (npages, page, Hkv, d)
        self.kc = torch.full(shape, float("nan"), dtype=DT[dtype])
        self.vc = torch.full(shape, float("nan"), dtype=DT[dtype])
        for i, n in enumerate(lens):
            for t in range(n):
                p = int(self.table[i, t // page])
                self.kc[p, t % page], self.vc[p, t % page] = self.k[i][t], self.v[i][t]
        self.lens, self.page = lens, page

    def cuda(self):
        return (self.kc.cuda(), self.vc.cuda(), self.table.cuda(),
                torch.tensor(self.lens, dtype=torch.int32, device="cuda"))


def _expect(c, q, i, window=0, sinks=0, scale=None):
    n = c.lens[i]
    if n == 0:
        z = np.zeros(q[i].shape)
        return z, z
    o, _, mag = attention(to64(q[i])[None, None], to64(c.k[i])[None], to64(c.v[i])[None],
                          window=window, sinks=sinks, scale=scale, magnitude=True)
    return o[0, 0], mag[0, 0]


def _check(c, q, o, dtype, **kw):
    u = unit(dtype)
    for i in range(len(c.lens)):
        ref, mag = _expect(c, q, i, **kw)
        close(to64(o[i]), ref, u * np.abs(ref) * (1 + 2 * u) + (u + 4 * F32) * mag + 1e-30,
              f"sequence {i} of {c.lens[i]} tokens")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_lengths(dtype, d, page):
    import gated_delta_rule_79_b200 as g
    c = Cache([0, 1, 2, 15, 16, 17, 63, 64, 65, 200, 513], 2, d, page, dtype)
    q = randn((11, 6, d), 5, dtype)
    o = g.attn_decode(q.cuda(), *c.cuda())
    _check(c, q, o, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (12, 4), (16, 1), (34, 2), (64, 1)])
def test_head_groups(dtype, Hq, Hkv):
    import gated_delta_rule_79_b200 as g
    c = Cache([300, 77], Hkv, 128, 32, dtype, seed=4)
    q = randn((2, Hq, 128), 6, dtype)
    _check(c, q, g.attn_decode(q.cuda(), *c.cuda(), scale=0.2), dtype, scale=0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (20, 0), (64, 4), (100, 70), (5000, 3)])
def test_window_reads_no_page_before_it(dtype, window, sinks):
    """Pages between the sinks and the window may have been given away: their entries are -1
    and must not be looked at (the status stays clean)."""
    import gated_delta_rule_79_b200 as g
    c = Cache([400, 3, 111], 2, 64, 16, dtype)
    for i, n in enumerate(c.lens):
        for pg in range(c.per):
            tokens = range(pg * 16, min(n, pg * 16 + 16))
            if not any(n - 1 - t < window or t < sinks for t in tokens):
                c.table[i, pg] = -1
    q = randn((3, 4, 64), 7, dtype)
    ws = torch.zeros(g.attn_decode_workspace_bytes(3, 4, 2, 64, 16, c.per, DT[dtype], window, sinks),
                     dtype=torch.uint8, device="cuda")
    o = g.attn_decode(q.cuda(), *c.cuda(), window=window, sinks=sinks, workspace=ws)
    g.workspace_status(ws)
    _check(c, q, o, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (20, 1)])
def test_stores_the_new_token(dtype, d, Hq, Hkv):
    import gated_delta_rule_79_b200 as g
    c = Cache([1, 16, 17, 250, 0], Hkv, d, 16, dtype, seed=3)
    q = randn((5, Hq, d), 8, dtype)
    kc, vc, table, lens = c.cuda()
    full_k, full_v = kc.clone(), vc.clone()
    knew, vnew = randn((5, Hkv, d), 1, dtype), randn((5, Hkv, d), 2, dtype)
    for i, n in enumerate(c.lens):
        if n:
            p = int(c.table[i, (n - 1) // 16])
            knew[i], vnew[i] = c.k[i][n - 1], c.v[i][n - 1]
            kc[p, (n - 1) % 16] = float("nan")
            vc[p, (n - 1) % 16] = float("nan")
    o = g.attn_decode(q.cuda(), kc, vc, table, lens, k=knew.cuda(), v=vnew.cuda())
    _check(c, q, o, dtype)
    # nothing else in the caches changed
    bits = {"bf16": torch.int16, "f32": torch.int32}[dtype]
    assert torch.equal(kc.view(bits), full_k.view(bits)) and torch.equal(vc.view(bits), full_v.view(bits))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv,d,extra", [
    ([1500, 3, 700], 4, 2, 128, 200),                        # a table far larger than its contents
    ([900] + [13 * i % 41 for i in range(69)], 2, 1, 64, 20),     # more sequences than lanes
    ([600, 0, 470] + [9 * i + 1 for i in range(17)], 8, 8, 128, 10),
    ([2100, 1500, 0, 7, 1024], 1184, 1, 128, 1),             # several rounds of CTAs: large parts
    ([i % 23 for i in range(1030)], 1, 1, 64, 0),            # too many sequences to be cut
])
def test_batches_that_are_cut_unevenly(dtype, lens, Hq, Hkv, d, extra):
    import gated_delta_rule_79_b200 as g
    c = Cache(lens, Hkv, d, 64, dtype, extra=extra, seed=6)
    N = len(lens)
    q, knew, vnew = randn((N, Hq, d), 9, dtype), randn((N, Hkv, d), 1, dtype), randn((N, Hkv, d), 2, dtype)
    for i, n in enumerate(lens):
        if n:
            p, r = int(c.table[i, (n - 1) // 64]), (n - 1) % 64
            knew[i], vnew[i] = c.k[i][n - 1], c.v[i][n - 1]
            c.kc[p, r], c.vc[p, r] = float("nan"), float("nan")
    kc, vc, table, t = c.cuda()
    ws = torch.zeros(g.attn_decode_workspace_bytes(N, Hq, Hkv, d, 64, c.per, DT[dtype]),
                     dtype=torch.uint8, device="cuda")
    o = g.attn_decode(q.cuda(), kc, vc, table, t, k=knew.cuda(), v=vnew.cuda(), workspace=ws)
    g.workspace_status(ws)
    _check(c, q, o, dtype)
    again = g.attn_decode(q.cuda(), kc, vc, table, t)           # the new tokens were stored
    assert torch.equal(o, again)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,Hq,Hkv,d,most", [(33, 8, 8, 128, 700), (37, 8, 8, 128, 331), (64, 4, 4, 64, 400),
                                             (2, 16, 16, 128, 1500), (12, 8, 8, 32, 640)])
def test_places_that_the_parts_fill(dtype, N, Hq, Hkv, d, most):
    """Batches that take one round of CTAs: the parts are the shortest that the places hold."""
    import gated_delta_rule_79_b200 as g
    lens = [most] + [(i * 7919 + 13) % most for i in range(1, N)]
    lens[-1] = 0
    c = Cache(lens, Hkv, d, 16, dtype, extra=40, seed=8)
    q = randn((N, Hq, d), 9, dtype)
    kc, vc, table, t = c.cuda()
    _check(c, q, g.attn_decode(q.cuda(), kc, vc, table, t), dtype)
    # the same tables with every sequence but the empty one cut to one length
    n = min(x for x in lens if x)
    c.lens = [min(x, n) for x in lens]
    c.k, c.v = [x[:n] for x in c.k], [x[:n] for x in c.v]
    _check(c, q, g.attn_decode(q.cuda(), kc, vc, table, t.clamp(max=n)), dtype)


def test_pages_and_lengths_outside_the_cache_are_left_out_and_reported():
    import gated_delta_rule_79_b200 as g
    c = Cache([100, 100, 100], 2, 128, 16, "bf16")
    q = randn((3, 4, 128), 9, "bf16")
    kc, vc, table, lens = c.cuda()
    table[1, 2] = 10 ** 6
    table[1, 3] = -7
    lens[2] = 10 ** 6
    table[2, 100 // 16:] = table[2, 0]
    ws = torch.zeros(g.attn_decode_workspace_bytes(3, 4, 2, 128, 16, c.per, torch.bfloat16),
                     dtype=torch.uint8, device="cuda")
    o = g.attn_decode(q.cuda(), kc, vc, table, lens, workspace=ws)
    with pytest.raises(g.GdrError) as e:
        g.workspace_status(ws)
    assert e.value.status == g.GDR_ERR_INVALID_ARG and "paged cache" in str(e.value)
    g.workspace_status(ws)                      # read once, then clean
    ref, mag = _expect(c, q, 0)
    close(to64(o[0]), ref, 2.0 ** -8 * 1.01 * (np.abs(ref) + mag) + F32, "the good sequence")
    keep = [t for t in range(100) if not 32 <= t < 64]
    ref, _, mag = attention(to64(q[1])[None, None], to64(c.k[1][keep])[None], to64(c.v[1][keep])[None],
                            magnitude=True)
    close(to64(o[1]), ref[0, 0], 2.0 ** -8 * 1.01 * (np.abs(ref) + mag)[0, 0] + F32, "without the pages")


def test_new_token_past_a_full_cache_is_left_out():
    import gated_delta_rule_79_b200 as g
    c = Cache([32, 20], 2, 64, 16, "bf16", extra=0)
    kc, vc, table, lens = c.cuda()
    before = kc.clone(), vc.clone()
    lens[0] = 33
    q, new = randn((2, 4, 64), 1, "bf16"), randn((2, 2, 64), 2, "bf16")
    ws = torch.zeros(g.attn_decode_workspace_bytes(2, 4, 2, 64, 16, c.per, torch.bfloat16),
                     dtype=torch.uint8, device="cuda")
    o = g.attn_decode(q.cuda(), kc, vc, table, lens, k=new.cuda(), v=new.cuda(), workspace=ws)
    with pytest.raises(g.GdrError):
        g.workspace_status(ws)
    ref, mag = _expect(c, q, 0)
    close(to64(o[0]), ref, 2.0 ** -8 * 1.01 * (np.abs(ref) + mag) + F32, "the 32 tokens it holds")
    p0, p1 = (table[0].long(), table[1].long())
    assert torch.equal(kc[p0], before[0][p0]) and torch.equal(vc[p0], before[1][p0])
    assert torch.equal(kc[p1[1], 3].cpu(), new[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 8, 128])
def test_append(dtype, page):
    import gated_delta_rule_79_b200 as g
    N, K, H, d = 4, 37, 3, 64
    per = 200 // page + 1
    table = torch.randperm(N * per).view(N, per).int().cuda()
    kc = torch.zeros(N * per, page, H, d, dtype=DT[dtype], device="cuda")
    vc = torch.zeros_like(kc)
    k, v = randn((N, K, H, d), 1, dtype).cuda(), randn((N, K, H, d), 2, dtype).cuda()
    start = torch.tensor([0, 5, 150, 99], dtype=torch.int32, device="cuda")
    counts = torch.tensor([37, 0, 20, 1], dtype=torch.int32, device="cuda")
    g.kv_append(k, v, kc, vc, table, start, counts)
    wk, wv = torch.zeros_like(kc), torch.zeros_like(vc)
    for n in range(N):
        for t in range(int(counts[n])):
            p = int(start[n]) + t
            wk[table[n, p // page].long(), p % page] = k[n, t]
            wv[table[n, p // page].long(), p % page] = v[n, t]
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    # outside the cache: skipped, recorded
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bad = table.clone()
    bad[0] = -1
    start = torch.tensor([0, per * page, -5, 0], dtype=torch.int32, device="cuda")
    counts = torch.tensor([37, 37, 5, 0], dtype=torch.int32, device="cuda")
    g.kv_append(k, v, kc, vc, bad, start, counts, workspace=ws)
    with pytest.raises(g.GdrError):
        g.workspace_status(ws)
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_run(dtype):
    """A padded batch of prompts prefilled with a window and sinks, its keys and values put into
    pages, then tokens decoded one by one: every output is that of attention over the whole."""
    import gated_delta_rule_79_b200 as g
    B, T, Hq, Hkv, d, page, new = 3, 90, 4, 2, 64, 16, 5
    kw = dict(window=40, sinks=2)
    lens = [90, 33, 1]
    q, k, v = (randn((B, T + new, h, d), s, dtype) for h, s in ((Hq, 1), (Hkv, 2), (Hkv, 3)))
    L = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qc, kcu, vcu = (x[:, :T].contiguous().cuda() for x in (q, k, v))
    o, _ = g.attn_prefill(qc, kcu, vcu, lengths=L, **kw)
    per = -(-(T + new) // page)
    table = torch.randperm(B * per).view(B, per).int().cuda()
    kc = torch.full((B * per, page, Hkv, d), float("nan"), dtype=DT[dtype], device="cuda")
    vc = kc.clone()
    g.kv_append(kcu, vcu, kc, vc, table, torch.zeros_like(L), L)
    u = unit(dtype)
    for s in range(new):
        L += 1
        pick = [(b, T + s) for b in range(B)]
        x = [torch.stack([y[b, t] for b, t in pick]).cuda() for y in (q, k, v)]
        one = g.attn_decode(x[0], kc, vc, table, L, k=x[1], v=x[2], **kw)
        for b in range(B):
            n = lens[b]
            kk = torch.cat([k[b, :n], k[b, T:T + s + 1]])
            vv = torch.cat([v[b, :n], v[b, T:T + s + 1]])
            ref, _, mag = attention(to64(q[b, T + s])[None, None], to64(kk)[None], to64(vv)[None],
                                    magnitude=True, **kw)
            close(to64(one[b]), ref[0, 0], (u * 1.01 + 4 * F32) * (np.abs(ref) + mag)[0, 0], f"token {s}")
    for b, n in enumerate(lens):
        ref, _, mag = attention(*(to64(y[b:b + 1, :n]) for y in (q, k, v)), magnitude=True, **kw)
        close(to64(o[b, :n]), ref[0], (u * 1.01 + 4 * F32) * (np.abs(ref) + mag)[0], "prompt")
        assert torch.count_nonzero(o[b, n:]) == 0


def test_streams_graphs_and_changing_lengths():
    """One captured step replayed while the lengths grow, beside eager calls on another stream."""
    import gated_delta_rule_79_b200 as g
    c = Cache([250, 40, 130], 2, 128, 16, "bf16")
    kc, vc, table, lens = c.cuda()
    kc, vc = torch.nan_to_num(kc), torch.nan_to_num(vc)
    q = randn((3, 8, 128), 2, "bf16").cuda()
    g.attn_decode(q, kc, vc, table, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = g.attn_decode(q, kc, vc, table, lens)
    side = torch.cuda.Stream()
    for grow in range(4):
        lens += 3
        torch.cuda.synchronize()
        graph.replay()
        e = g.attn_decode(q, kc, vc, table, lens, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o, e)


def test_long_cache_past_32_bit_offsets():
    """A pool of more than 2^31 elements: a sequence whose pages lie at its far end."""
    import gated_delta_rule_79_b200 as g
    page, H, d = 128, 8, 128
    npages = (1 << 31) // (page * H * d) + 40
    kc = torch.zeros(npages, page, H, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    n = 3000
    table = torch.arange(npages - 1, npages - 1 - 24, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    k, v = randn((1, n, H, d), 1, "bf16"), randn((1, n, H, d), 2, "bf16")
    g.kv_append(k.cuda(), v.cuda(), kc, vc, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = randn((1, 16, d), 3, "bf16")
    o = g.attn_decode(q.cuda(), kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"))
    ref, _, mag = attention(to64(q)[:, None], to64(k), to64(v), magnitude=True)
    close(to64(o[0]), ref[0, 0], 2.0 ** -8 * 1.01 * (np.abs(ref) + mag)[0, 0] + F32, "o")

"""The linear-attention and softmax-attention mixers as measured calls.

Beside the gated delta rule the library has two more kinds of token mixer: linear attention
with one decay per head (``lin_prefill``, ``lin_decode``, ``lin_backward``) and softmax
attention with a sliding window and a few first tokens that stay visible (``attn_prefill``,
``attn_backward``, ``attn_decode`` over a paged key-value cache).  ``run`` computes a case
either through those entry points (``own``) or in plain torch operations in 32 bits;
``exact`` computes it from the definitions in 64 bits.

Definitions (one (batch, head) at a time, tokens t = 0 .. T-1):

    linear     S_t = decay S_{t-1} + v_t k_t^T,   o_t = S_t q_t
    softmax    o_i = sum_j p_ij v_j,   p_ij = exp(scale q_i.k_j) / sum over the visible j,
               query i sits at position p = Tk - Tq + i and sees key j when j <= p, both lie
               before the sequence's length, and p - j < window or j < sinks
               (window 0: every j <= p); a query that sees nothing gives 0
"""

import math

import torch

own = False

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one user's next token through one layer of 32 heads: latency
        dict(name="lin_decode_one", op="lin_decode", dtype="bf16", N=1, H=32, dk=128, dv=128),
        # the batched decode shapes of the gated delta rule's own benchmark (1 GB of state)
        dict(name="lin_decode_batch", op="lin_decode", dtype="bf16", N=256, H=32, dk=128, dv=128),
        # one prompt of 4096 tokens, 32 heads (the benchmark's prefill shapes)
        dict(name="lin_prefill_4k", op="lin_prefill", dtype="bf16", B=1, T=4096, H=32, dk=128,
             dv=128, state=False),
        # a batch of long prompts that continue from a carried state
        dict(name="lin_prefill_long", op="lin_prefill", dtype="bf16", B=4, T=16384, H=32, dk=128,
             dv=128, state=True),
        # training step of one layer at the benchmark's backward shapes
        dict(name="lin_backward_4k", op="lin_backward", dtype="bf16", B=1, T=4096, H=32, dk=128,
             dv=128, state=True),
        # fp32 training, odd length, unequal head sizes
        dict(name="lin_backward_f32", op="lin_backward", dtype="f32", B=2, T=1337, H=6, dk=64,
             dv=128, state=True),
        # sliding-window layer over a prompt: window 4096 with four sinks, grouped heads
        dict(name="attn_prefill_8k", op="attn_prefill", dtype="bf16", B=1, Tq=8192, Tk=8192, Hq=32,
             Hkv=8, d=128, window=4096, sinks=4, ragged=False),
        # the next part of padded prompts against what came before, odd window
        dict(name="attn_prefill_part", op="attn_prefill", dtype="bf16", B=3, Tq=500, Tk=2777, Hq=12,
             Hkv=4, d=64, window=1000, sinks=3, ragged=True),
        # training step of one sliding-window layer: forward and gradients
        dict(name="attn_train_4k", op="attn_train", dtype="bf16", B=1, Tq=4096, Tk=4096, Hq=16,
             Hkv=4, d=128, window=1024, sinks=4, ragged=False),
        # fp32 training of a padded batch with full causal attention, no grouping
        dict(name="attn_train_f32", op="attn_train", dtype="f32", B=3, Tq=777, Tk=777, Hq=6,
             Hkv=6, d=64, window=0, sinks=0, ragged=True),
        # one user's next token against a short cache: latency
        dict(name="attn_decode_one", op="attn_decode", dtype="bf16", N=1, Tmax=2000, page=16, Hq=32,
             Hkv=8, d=128, window=0, sinks=0),
        # a serving batch with caches of every length up to 16384
        dict(name="attn_decode_batch", op="attn_decode", dtype="bf16", N=64, Tmax=16384, page=64,
             Hq=32, Hkv=8, d=128, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lin_decode", "lin_prefill", "lin_backward", "attn_prefill", "attn_train",
                     "attn_decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("lin_"):
        dk, dv = rng.choice([(32, 32), (64, 64), (128, 128), (128, 128), (128, 64), (64, 128)])
        H = rng.choice([1, 3, 4, 8, 16, 32])
        if op == "lin_decode":
            return dict(op=op, dtype=dtype, N=_log(rng, 1, 256), H=H, dk=dk, dv=dv)
        most = 1 << (21 if dtype == "bf16" else 17) if op == "lin_prefill" else \
            1 << (17 if dtype == "bf16" else 15)
        B = rng.choice([1, 1, 2, 3, 4])
        T = _log(rng, 1, max(2, min(16384, most // (B * H))))
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, dk=dk, dv=dv, state=rng.random() < 0.6)
    d = rng.choice([32, 64, 64, 128, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    # a gradient through queries that see one key only is 0: training sees more
    few = 8 if op == "attn_train" else 1
    window = rng.choice([0, _log(rng, few, 4096)])
    sinks = rng.choice([0, rng.randint(1, 8)]) if window else 0
    if op == "attn_decode":
        N = _log(rng, 1, 128)
        Tmax = _log(rng, 1, max(2, min(65536, (1 << 22) // (N * Hkv))))
        return dict(op=op, dtype=dtype, N=N, Tmax=Tmax, page=rng.choice([1, 16, 32, 64, 128]),
                    Hq=Hq, Hkv=Hkv, d=d, window=window, sinks=sinks)
    most = {("attn_prefill", "bf16"): 30, ("attn_prefill", "f32"): 26, ("attn_train", "bf16"): 27,
            ("attn_train", "f32"): 24}[op, dtype]
    B = rng.choice([1, 1, 2, 3])
    Tk = _log(rng, few, min(8192, max(16, int(math.sqrt((1 << most) / (B * Hq))))))
    Tq = Tk if op == "attn_train" or rng.random() < 0.6 else rng.randint(1, Tk)
    return dict(op=op, dtype=dtype, B=B, Tq=Tq, Tk=Tk, Hq=Hq, Hkv=Hkv, d=d, window=window,
                sinks=sinks, ragged=rng.random() < 0.4)


# ---- inputs -------------------------------------------------------------------------------

def _spread(n, most):
    """n lengths from 1 to `most`, the first of them `most`, the others spread evenly."""
    return [max(1, most - int(most * ((i * 0.6180339887) % 1.0))) for i in range(n)]


def _decays(H, dev):
    """One decay per head from 1 - 2^-4 (a memory of 16 tokens) to 1 - 2^-11, the spacing that
    such mixers use."""
    e = 4 + 7 * torch.arange(H, dtype=torch.float64, device=dev) / max(1, H - 1)
    return (1 - torch.exp2(-e)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    t = _T[case["dtype"]]

    def normal(*shape, dtype=t, std=1.0):
        x = torch.randn(shape, generator=g, device=dev, dtype=dtype)
        return x.mul_(std) if std != 1.0 else x

    op, s = case["op"], dict(case)
    if op.startswith("lin_"):
        dk, dv, H = case["dk"], case["dv"], case["H"]
        lead = (case["N"], H) if op == "lin_decode" else (case["B"], case["T"], H)
        # q carries the 1/sqrt(d_k) of the projection before it
        s["q"] = normal(*lead, dk, std=dk ** -0.5)
        s["k"] = normal(*lead, dk)
        s["v"] = normal(*lead, dv)
        s["decay"] = _decays(H, dev)
        if op == "lin_decode":
            s["S"] = normal(case["N"], H, dv, dk, dtype=torch.float32)
            return s
        state = (case["B"], H, dv, dk)
        s["s0"] = normal(*state, dtype=torch.float32) if case["state"] else None
        if op == "lin_backward":
            s["do"] = normal(*lead, dv)
            s["dsf"] = normal(*state, dtype=torch.float32) if case["state"] else None
        return s
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    if op == "attn_decode":
        N, page = case["N"], case["page"]
        lens = _spread(N, case["Tmax"])
        per = -(-case["Tmax"] // page)
        s["q"] = normal(N, Hq, d)
        s["k"] = normal(N, Hkv, d)
        s["v"] = normal(N, Hkv, d)
        # pages in no order, as an allocator hands them out
        s["table"] = torch.randperm(N * per, generator=g, device=dev).to(torch.int32).view(N, per)
        s["kc"] = normal(N * per, page, Hkv, d)
        s["vc"] = normal(N * per, page, Hkv, d)
        s["lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        return s
    B = case["B"]
    s["q"] = normal(B, case["Tq"], Hq, d)
    s["k"] = normal(B, case["Tk"], Hkv, d)
    s["v"] = normal(B, case["Tk"], Hkv, d)
    s["lengths"] = torch.tensor(_spread(B, case["Tk"]), dtype=torch.int32, device=dev) \
        if case["ragged"] else None
    if op == "attn_train":
        s["do"] = normal(B, case["Tq"], Hq, d)
    return s


# ---- the plain form -------------------------------------------------------------------------

_C = 128


def _powers(log_decay, n):
    """exp(n log decay) for whole n >= 0 (a tensor broadcast against the heads), 0 where n < 0."""
    return torch.where(n < 0, 0.0, torch.exp(n.clamp(min=0).double() * log_decay)).float()


def _scan(q, k, v, decay, s0, first):
    """o_t = sum_{j<=t} decay^(t-j) (q_t.k_j) v_j + decay^(t+first) S0 q_t, chunk by chunk but
    all chunks at once, and the state decay^(T-1+first) S0 + decay^(1-first) * (sum of what the
    T tokens left, decayed to the last).  q, k [B, T, H, dk], v [B, T, H, dv]."""
    B, T, H, dk = q.shape
    dv, dev = v.shape[-1], q.device
    n = -(-T // _C)
    ld = torch.log(decay.double())

    def chunks(x):
        x = x.float().transpose(1, 2)
        return torch.nn.functional.pad(x, (0, 0, 0, n * _C - T)).view(B, H, n, _C, -1)

    q, k, v = chunks(q), chunks(k), chunks(v)
    t = torch.arange(_C, device=dev)
    D = _powers(ld[:, None, None], (t[:, None] - t[None, :])[None])
    o = ((q @ k.transpose(-1, -2)) * D[None, :, None]) @ v
    left = v.transpose(-1, -2) @ (k * _powers(ld[:, None], (_C - 1 - t)[None])[None, :, None, :, None])
    c = torch.arange(n, device=dev)
    W = _powers(ld[:, None, None], ((c[:, None] - 1 - c[None, :]) * _C)[None])
    enter = (W[None] @ left.view(B, H, n, dv * dk)).view(B, H, n, dv, dk)
    o += (q @ enter.transpose(-1, -2)) * _powers(ld[:, None], (t + 1)[None])[None, :, None, :, None]
    at = torch.arange(n * _C, device=dev).view(n, _C)
    if s0 is not None:
        o += (q @ s0.transpose(-1, -2)[:, :, None]) * \
            _powers(ld[:, None, None], (at + first)[None])[None, ..., None]
    w = _powers(ld[:, None, None], (T - first - at)[None])[None, ..., None] * (at < T)[..., None]
    end = v.reshape(B, H, n * _C, dv).transpose(-1, -2) @ (k * w).reshape(B, H, n * _C, dk)
    if s0 is not None:
        end = end + s0 * _powers(ld, torch.full_like(ld, T))[:, None, None]
    return o.reshape(B, H, n * _C, dv)[:, :, :T].transpose(1, 2), end


def _lin_plain(s):
    t = s["q"].dtype
    if s["op"] == "lin_decode":
        S = s["S"]
        S.mul_(s["decay"][:, None, None]).add_(s["v"].float()[..., None] * s["k"].float()[..., None, :])
        return {"o": (S @ s["q"].float()[..., None])[..., 0].to(t), "state": S}
    if s["op"] == "lin_prefill":
        o, end = _scan(s["q"], s["k"], s["v"], s["decay"], s["s0"], 1)
        return {"o": o.to(t).contiguous(), "state": end}
    q, k, v, do = s["q"], s["k"], s["v"], s["do"]
    turned = None if s["s0"] is None else s["s0"].transpose(-1, -2)
    dq, _ = _scan(do, v, k, s["decay"], turned, 1)
    q, k, v, do = q.flip(1), k.flip(1), v.flip(1), do.flip(1)
    dv, ds0 = _scan(k, q, do, s["decay"], s["dsf"], 0)
    turned = None if s["dsf"] is None else s["dsf"].transpose(-1, -2)
    dk, _ = _scan(v, do, q, s["decay"], turned, 0)
    return {"dq": dq.to(t).contiguous(), "dk": dk.flip(1).to(t), "dv": dv.flip(1).to(t), "ds0": ds0}


def _visible(Tq, Tk, window, sinks, lengths, dev):
    """[B or 1, 1, 1, Tq, Tk] truth values."""
    p = torch.arange(Tk - Tq, Tk, device=dev)[:, None]
    j = torch.arange(Tk, device=dev)[None, :]
    m = j <= p
    if window:
        m &= (p - j < window) | (j < sinks)
    m = m[None]
    if lengths is not None:
        m = m & (j[None] < lengths[:, None, None]) & (p[None] < lengths[:, None, None])
    return m[:, None, None]


def _attn_forward(s):
    B, Tq, Hq, d = s["q"].shape
    Tk, Hkv = s["k"].shape[1:3]
    q = s["q"].float().view(B, Tq, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4)
    k = s["k"].float().permute(0, 2, 1, 3)[:, :, None]
    v = s["v"].float().permute(0, 2, 1, 3)[:, :, None]
    sees = _visible(Tq, Tk, s["window"], s["sinks"], s["lengths"], q.device)
    p = ((q * d ** -0.5) @ k.transpose(-1, -2)).masked_fill_(~sees, -math.inf)
    m = p.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = p.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    p = p.div_(torch.where(l == 0, 1.0, l))
    return q, k, v, p, p @ v, (m0 + torch.log(l))[..., 0]


def _heads_last(x, t):
    """[B, Hkv, G, T, d] to [B, T, Hkv * G, d]."""
    B, Hkv, G, T, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(B, T, Hkv * G, d).to(t)


def _attn_plain(s):
    t, d = s["q"].dtype, s["d"]
    if s["op"] == "attn_decode":
        N, Hq = s["N"], s["Hq"]
        Hkv, page, lens = s["Hkv"], s["page"], s["lengths"].long()
        at = lens - 1
        where = s["table"].long().gather(1, (at // page)[:, None])[:, 0]
        s["kc"][where, at % page] = s["k"]
        s["vc"][where, at % page] = s["v"]
        k = s["kc"][s["table"].long()].view(N, -1, Hkv, d).permute(0, 2, 1, 3).float()
        v = s["vc"][s["table"].long()].view(N, -1, Hkv, d).permute(0, 2, 1, 3).float()
        j = torch.arange(k.shape[2], device=k.device)[None]
        sees = j < lens[:, None]
        if s["window"]:
            sees &= (at[:, None] - j < s["window"]) | (j < s["sinks"])
        q = s["q"].float().view(N, Hkv, Hq // Hkv, d) * d ** -0.5
        p = (q @ k.transpose(-1, -2)).masked_fill_(~sees[:, None, None], -math.inf)
        p = torch.exp(p - p.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        return {"o": o.view(N, Hq, d).to(t), "k_cache": s["kc"], "v_cache": s["vc"]}
    q, k, v, p, o, lse = _attn_forward(s)
    B, Hkv, G, Tq, _ = q.shape
    got = {"o": _heads_last(o, t), "lse": lse.reshape(B, Hkv * G, Tq)}
    if s["op"] == "attn_train":
        do = s["do"].float().view(B, Tq, Hkv, G, d).permute(0, 2, 3, 1, 4)
        got["dv"] = (p.transpose(-1, -2) @ do).sum(2).transpose(1, 2).to(t).contiguous()
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) * d ** -0.5
        got["dq"] = _heads_last(ds @ k, t)
        got["dk"] = (ds.transpose(-1, -2) @ q).sum(2).transpose(1, 2).to(t).contiguous()
    return got


# ---- one pass -------------------------------------------------------------------------------

def _own(s):
    import gated_delta_rule_79_b200 as g
    op = s["op"]
    if op == "lin_decode":
        return {"o": g.lin_decode(s["q"], s["k"], s["v"], s["decay"], s["S"]), "state": s["S"]}
    if op == "lin_prefill":
        o, end = g.lin_prefill(s["q"], s["k"], s["v"], s["decay"], s["s0"])
        return {"o": o, "state": end}
    if op == "lin_backward":
        dq, dk, dv, ds0 = g.lin_backward(s["q"], s["k"], s["v"], s["decay"], s["s0"], s["do"], s["dsf"])
        return {"dq": dq, "dk": dk, "dv": dv, "ds0": ds0}
    if op == "attn_decode":
        o = g.attn_decode(s["q"], s["kc"], s["vc"], s["table"], s["lengths"], k=s["k"], v=s["v"],
                          window=s["window"], sinks=s["sinks"])
        return {"o": o, "k_cache": s["kc"], "v_cache": s["vc"]}
    how = dict(window=s["window"], sinks=s["sinks"], lengths=s["lengths"])
    o, lse = g.attn_prefill(s["q"], s["k"], s["v"], **how)
    got = {"o": o, "lse": lse}
    if op == "attn_train":
        got["dq"], got["dk"], got["dv"] = g.attn_backward(s["q"], s["k"], s["v"], o, lse, s["do"], **how)
    return got


def run(state):
    if own:
        return _own(state)
    return _lin_plain(state) if state["op"].startswith("lin_") else _attn_plain(state)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("lin_"):
        dk, dv = case["dk"], case["dv"]
        if op == "lin_decode":
            heads = case["N"] * case["H"]
            return {"bytes": heads * (8 * dk * dv + e * 2 * (dk + dv)), "flops": heads * 5 * dk * dv}
        heads = case["B"] * case["H"]
        states = 4 * dk * dv * heads
        rows = heads * case["T"]
        if op == "lin_prefill":
            return {"bytes": rows * e * 2 * (dk + dv) + states * (2 if case["state"] else 1),
                    "flops": rows * 4 * dk * dv}
        # S is rebuilt for dq, and its gradient gives dk, dv
        return {"bytes": rows * e * (4 * dk + 3 * dv) + states * (3 if case["state"] else 1),
                "flops": rows * 10 * dk * dv}
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    window, sinks = case["window"], case["sinks"]

    def seen(p):
        if not window or p + 1 <= window:
            return p + 1
        return window + min(sinks, p + 1 - window)

    if op == "attn_decode":
        keys = sum(seen(n - 1) for n in _spread(case["N"], case["Tmax"]))
        return {"bytes": e * d * (2 * Hkv * keys + case["N"] * (2 * Hq + 4 * Hkv)),
                "flops": 4 * d * Hq * keys}
    B, Tq, Tk = case["B"], case["Tq"], case["Tk"]
    lens = _spread(B, Tk) if case["ragged"] else [Tk] * B
    pairs = sum(seen(p) for n in lens for p in range(Tk - Tq, n)) * Hq
    q, kv = B * Tq * Hq * d * e, B * Tk * Hkv * d * e
    if op == "attn_prefill":
        return {"bytes": 2 * q + 2 * kv + 4 * B * Tq * Hq, "flops": 4 * d * pairs}
    return {"bytes": 5 * q + 6 * kv + 8 * B * Tq * Hq, "flops": 14 * d * pairs}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    if op == "lin_decode":
        S = s["decay"].to(f).view(1, -1, 1, 1) * s["S"].to(f)
        S = S + torch.einsum("nhv,nhk->nhvk", s["v"].to(f), s["k"].to(f))
        return {"o": torch.einsum("nhvk,nhk->nhv", S, s["q"].to(f)), "state": S}
    if op.startswith("lin_"):
        # every pair of tokens of a head at once: M[t, j] = decay^(t-j) for j <= t
        B, T, H, dk = s["q"].shape
        dv = case["dv"]
        dev = s["q"].device
        t = torch.arange(T, device=dev, dtype=f)
        gap = t[:, None] - t[None, :]
        out = {n: torch.empty(B, T, H, w, dtype=f, device=dev)
               for n, w in ((("o", dv),) if op == "lin_prefill" else (("dq", dk), ("dk", dk), ("dv", dv)))}
        end = torch.empty(B, H, dv, dk, dtype=f, device=dev)
        for h in range(H):
            a = float(s["decay"][h])
            M = torch.pow(torch.tensor(a, dtype=f, device=dev), gap.clamp(min=0)).tril_()
            up, down = a ** (t + 1), a ** (T - 1 - t)
            for b in range(B):
                q, k, v = (s[n][b, :, h].to(f) for n in "qkv")
                S = s["s0"][b, h].to(f) if s["s0"] is not None else torch.zeros(dv, dk, dtype=f, device=dev)
                if op == "lin_prefill":
                    A = (q @ k.T).mul_(M)
                    out["o"][b, :, h] = A @ v + up[:, None] * (q @ S.T)
                    end[b, h] = a ** T * S + v.T @ (down[:, None] * k)
                    continue
                do = s["do"][b, :, h].to(f)
                F = s["dsf"][b, h].to(f) if s["dsf"] is not None else torch.zeros_like(S)
                A = (do @ v.T).mul_(M)
                out["dq"][b, :, h] = A @ k + up[:, None] * (do @ S)
                out["dk"][b, :, h] = A.T @ q + down[:, None] * (v @ F)
                A = (q @ k.T).mul_(M)
                out["dv"][b, :, h] = A.T @ do + down[:, None] * (k @ F.T)
                end[b, h] = a ** T * F + do.T @ (up[:, None] * q)
        out["state" if op == "lin_prefill" else "ds0"] = end
        return out
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    window, sinks = case["window"], case["sinks"]
    lens = [int(x) for x in s["lengths"]] if s["lengths"] is not None else [case["Tk"]] * case["B"]
    dev = s["q"].device
    if op == "attn_decode":
        o = torch.zeros(case["N"], Hq, d, dtype=f, device=dev)
        for n, L in enumerate(lens):
            pages = s["table"][n, : -(-L // case["page"])].long()
            k = s["kc"][pages].reshape(-1, Hkv, d)[:L].to(f)
            v = s["vc"][pages].reshape(-1, Hkv, d)[:L].to(f)
            k[L - 1], v[L - 1] = s["k"][n].to(f), s["v"][n].to(f)
            if window and L > window:
                keep = torch.cat([torch.arange(min(sinks, L - window), device=dev),
                                  torch.arange(L - window, L, device=dev)])
                k, v = k[keep], v[keep]
            q = s["q"][n].to(f).view(Hkv, G, d)
            w = torch.softmax(torch.einsum("hgd,jhd->hgj", q, k) / math.sqrt(d), -1)
            o[n] = torch.einsum("hgj,jhd->hgd", w, v).reshape(Hq, d)
        return {"o": o, "k_cache": None, "v_cache": None}
    B, Tq, Tk = case["B"], case["Tq"], case["Tk"]
    o = torch.zeros(B, Tq, Hq, d, dtype=f, device=dev)
    lse = torch.full((B, Hq, Tq), -math.inf, dtype=f, device=dev)
    got = {"o": o, "lse": lse}
    if op == "attn_train":
        got["dq"] = torch.zeros_like(o)
        got["dk"] = torch.zeros(B, Tk, Hkv, d, dtype=f, device=dev)
        got["dv"] = torch.zeros_like(got["dk"])
    first = Tk - Tq
    for b, L in enumerate(lens):
        rows = max(0, L - first)            # queries before the length
        if not rows:
            continue
        i = torch.arange(first, first + rows, device=dev)
        j = torch.arange(L, device=dev)
        hide = j[None] > i[:, None]
        if window:
            hide |= (j[None] <= i[:, None] - window) & (j[None] >= sinks)
        for h in range(Hq):
            q, k, v = s["q"][b, :rows, h].to(f), s["k"][b, :L, h // G].to(f), s["v"][b, :L, h // G].to(f)
            x = (q @ k.T / math.sqrt(d)).masked_fill_(hide, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[:, None])
            o[b, :rows, h], lse[b, h, :rows] = w @ v, z
            if op == "attn_train":
                do = s["do"][b, :rows, h].to(f)
                dw = do @ v.T
                dx = w * (dw - (w * dw).sum(-1, keepdim=True)) / math.sqrt(d)
                got["dq"][b, :rows, h] = dx @ k
                got["dk"][b, :L, h // G] += dx.T @ q
                got["dv"][b, :L, h // G] += w.T @ do
    return got

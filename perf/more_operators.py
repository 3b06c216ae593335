"""Operators around windows, shared prefixes and normed heads, in plain torch and as the library's calls.

``window``        causal attention of which a query sees its last `window` keys and the first `sinks`
                  (forward, and ``window_grad``: its gradients), query heads sharing key/value heads
``paged_window``  the same over a paged key/value cache, chunks or one token a sequence
``paged_prefix``  attention over a paged cache whose sequences share a prefix group by group
``norm_rope``     each head's row normed and rotated in one pass (``norm_rope_grad``: its gradients)
``append_norm``   new tokens' keys (normed and rotated) and values into their pages, queries beside them

A cache is a pair [P, Hkv, S, d] of key and value pages, a table int32 [B, M] of page numbers (-1:
none) and int32 lengths; sequence b's token t lies in slot t % S of page table[b, t // S].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # the 1000-length configuration with a narrow window: latency counts
        dict(name="window_small", op="window", dtype="fp16", b=2, h=8, hkv=4, n=1000, d=64, window=200, sinks=3),
        # the 16384-length configuration, shared heads: a training step's or a prompt's forward pass
        dict(name="window_long", op="window", dtype="bf16", b=1, h=32, hkv=8, n=16384, d=128, window=4096, sinks=4),
        # the gradients of a small step, an odd window and no sinks
        dict(name="window_grad_small", op="window_grad", dtype="fp16", b=2, h=8, hkv=8, n=1000, d=64, window=333,
             sinks=0),
        # the gradients at the 4096-length configuration, heads shared by four
        dict(name="window_grad", op="window_grad", dtype="bf16", b=4, h=16, hkv=4, n=4096, d=128, window=1024,
             sinks=4),
        # a serving batch: one token each, contexts far longer than the window
        dict(name="window_decode", op="paged_window", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=64,
             q_min=1, q_max=1, kv_min=2000, kv_max=32768, window=2048, sinks=4, mix=1),
        # a mixed step: chunks of a few to some hundred tokens
        dict(name="window_chunk", op="paged_window", dtype="bf16", hq=20, hkv=4, d=128, page=32, seqs=12,
             q_min=1, q_max=1024, kv_min=1500, kv_max=16384, window=1024, sinks=16, mix=2),
        # a few samples of one prompt: one token each, latency counts
        dict(name="prefix_decode_small", op="paged_prefix", dtype="bf16", hq=32, hkv=8, d=128, page=16, groups=1,
             seqs=8, q_min=1, q_max=1, prefix_min=2000, prefix_max=2000, own_min=10, own_max=200, mix=3),
        # many requests behind two long system prompts
        dict(name="prefix_decode", op="paged_prefix", dtype="bf16", hq=32, hkv=8, d=128, page=16, groups=2,
             seqs=64, q_min=1, q_max=1, prefix_min=8000, prefix_max=16384, own_min=20, own_max=2000, mix=4),
        # several tokens a sequence (drafts looked over) behind a very long document, small heads
        dict(name="prefix_chunk", op="paged_prefix", dtype="fp16", hq=16, hkv=4, d=64, page=64, groups=1,
             seqs=24, q_min=2, q_max=40, prefix_min=65536, prefix_max=65536, own_min=50, own_max=1500, mix=5),
        # queries of a training step at the 4096-length configuration
        dict(name="norm_rope_train", op="norm_rope", dtype="bf16", b=4, h=16, n=4096, d=128, rotary=128,
             interleaved=False, start=0),
        # their gradient
        dict(name="norm_rope_grad", op="norm_rope_grad", dtype="bf16", b=4, h=16, n=4096, d=128, rotary=128,
             interleaved=False, start=0),
        # a decoding step's new tokens
        dict(name="append_norm_step", op="append_norm", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=64,
             q_min=1, q_max=1, kv_min=1000, kv_max=8192, rotary=128, interleaved=False, mix=6),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], its logarithm spread evenly where the range is wide."""
    if hi <= 10 * lo:
        return rng.randint(lo, hi)
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _range(rng, name, lo, hi):
    a, b = sorted((_spread(rng, lo, hi), _spread(rng, lo, hi)))
    return {name + "_min": a, name + "_max": b}


def draw(rng):
    mix = rng.randrange(1 << 30)
    op = rng.choice(["window", "window_grad", "paged_window", "paged_prefix", "norm_rope", "norm_rope_grad",
                     "append_norm"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    if op in ("window", "window_grad"):
        grad = op == "window_grad"
        n, window = _spread(rng, 100, 16384), _spread(rng, 16, 4096)
        case = dict(op=op, dtype=dtype, b=_spread(rng, 1, 4), h=hkv * group, hkv=hkv, n=n,
                    d=rng.choice([64, 128]) if grad else d, window=window,
                    sinks=rng.choice([0, 0, 1, 4, 16, 130]))
        while case["b"] * case["h"] * n * min(n, window + 1024) * case["d"] > 1 << (34 if grad else 36):
            if case["b"] > 1:
                case["b"] = 1
            else:
                hkv = max(1, hkv // 2)
                group = group if hkv > 1 else max(1, group // 2)
                case["hkv"], case["h"] = hkv, hkv * group
                if case["h"] == 1:
                    break
        return case
    if op in ("norm_rope", "norm_rope_grad"):
        b, h, n = _spread(rng, 1, 8), rng.randint(1, 32), _spread(rng, 100, 8192)
        h = max(1, min(h, (1 << 25) // (b * n * d)))
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), b=b, h=h, n=n, d=d,
                    rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.5,
                    start=_spread(rng, 1, 1 << 20))
    if op == "append_norm":
        case = dict(op=op, dtype=dtype, hq=hkv * group, hkv=hkv, d=d, page=page, seqs=_spread(rng, 1, 64),
                    **_range(rng, "q", 1, 1024), **_range(rng, "kv", 1100, 8192),
                    rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.5, mix=mix)
        while sum(_lengths(case)[0]) * (group + 2) * hkv * d > 1 << 24:
            case["q_min"], case["q_max"] = max(1, case["q_min"] // 2), max(1, case["q_max"] // 2)
        return case
    single = rng.random() < 0.5
    if op == "paged_window":
        q = dict(q_min=1, q_max=1) if single else _range(rng, "q", 1, 1024)
        case = dict(op=op, dtype=dtype, hq=hkv * group, hkv=hkv, d=d, page=page, seqs=_spread(rng, 1, 64), **q,
                    **_range(rng, "kv", q["q_max"], 16384), window=_spread(rng, 16, 4096),
                    sinks=rng.choice([0, 1, 4, 64]), mix=mix)
        # the plain form pads every sequence to the longest: bounded in scores and in pages
        while case["seqs"] > 1 and (case["seqs"] * case["hq"] * case["q_max"] * case["kv_max"] > 1 << 31
                                    or case["seqs"] * case["kv_max"] * hkv * d > 1 << 28):
            case["seqs"] = max(1, case["seqs"] // 2)
        return case
    q = dict(q_min=1, q_max=1) if single else _range(rng, "q", 1, 64)
    groups = rng.randint(1, 4)
    case = dict(op=op, dtype=dtype, hq=hkv * group, hkv=hkv, d=d, page=page, groups=groups,
                seqs=max(groups, _spread(rng, 1, 64)), **q, **_range(rng, "prefix", 300, 32768),
                **_range(rng, "own", q["q_max"], 2000), mix=mix)
    while case["seqs"] > groups and (
            case["seqs"] * case["hq"] * case["q_max"] * (case["prefix_max"] + case["own_max"]) > 1 << 31
            or case["seqs"] * (case["prefix_max"] + case["own_max"]) * hkv * d > 1 << 28):
        case["seqs"] = max(groups, case["seqs"] // 2)
    return case


def _lengths(case):
    """New tokens and lengths (new tokens among them) of each sequence: (q, kv)."""
    rng = random.Random(case["mix"])
    q = [_spread(rng, case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    q[0] = case["q_max"]
    if case["op"] == "paged_prefix":
        first, prefix = _groups(case)
        own_lens = [max(_spread(rng, case["own_min"], case["own_max"]), n) for n in q]
        own_lens[-1] = max(case["own_max"], q[-1])
        return q, [prefix[g] + own_lens[b] for g in range(case["groups"]) for b in range(first[g], first[g + 1])]
    kv = [max(_spread(rng, case["kv_min"], case["kv_max"]), n) for n in q]
    kv[-1] = max(case["kv_max"], q[-1])
    kv[0] = max(kv[0], q[0])
    return q, kv


def _groups(case):
    """Where each group's sequences begin (and the last one's end), and the tokens that a group shares: whole pages."""
    rng = random.Random(case["mix"] + 1)
    inner = sorted(rng.sample(range(1, case["seqs"]), case["groups"] - 1))
    lens = [_spread(rng, case["prefix_min"], case["prefix_max"]) for _ in range(case["groups"])]
    lens[0] = case["prefix_max"]
    return [0] + inner + [case["seqs"]], [n // case["page"] * case["page"] for n in lens]


def _inv_freq(case):
    return [10000.0 ** (-2.0 * i / case["rotary"]) for i in range(case["rotary"] // 2)]


def _first_key(case, i):
    """The first key of query i's window."""
    return max(0, i - case["window"] + 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d = DTYPES[case["dtype"]], case["d"]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std + mean).to(dtype)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    st = {"case": case}
    if "rotary" in case:
        st["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device="cuda")
    if case["op"] in ("window", "window_grad"):
        b, h, n = case["b"], case["h"], case["n"]
        st["q"], st["k"], st["v"] = normal(b, h, n, d), normal(b, case["hkv"], n, d), normal(b, case["hkv"], n, d)
        if case["op"] == "window_grad":
            # what the forward pass left, and the gradient that comes back
            st["do"] = normal(b, h, n, d)
            out = _plain_window(st)
            st["o"], st["lse"] = out["o"], out["lse"]
        return st
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        b, h, n = case["b"], case["h"], case["n"]
        # rows of different sizes, as a projection's heads have
        st["x"] = (normal(b, h, n, d, dtype=torch.float32)
                   * normal(b, h, n, 1, std=0.5, dtype=torch.float32).exp()).to(dt)
        st["weight"] = normal(d, std=0.2, mean=1.0)
        st["positions"] = torch.arange(case["start"], case["start"] + n, dtype=torch.int32, device="cuda")
        if case["op"] == "norm_rope_grad":
            st["dy"] = normal(b, h, n, d)
        return st
    # a cache whose pages lie in no order, some of them nobody's; a group's sequences share their first pages
    q, kv = _lengths(case)
    S, B = case["page"], case["seqs"]
    counts = [-(-n // S) for n in kv]
    shared, leader = [0] * B, list(range(B))
    if case["op"] == "paged_prefix":
        first, prefix = _groups(case)
        for i in range(case["groups"]):
            for b in range(first[i], first[i + 1]):
                leader[b], shared[b] = first[i], prefix[i] // S
        st["cu_groups"], st["prefix_lens"] = ints(first), ints(prefix)
    used = sum(n - (s if a != b else 0) for b, (n, s, a) in enumerate(zip(counts, shared, leader)))
    P, width = used + max(4, used // 16), max(counts)
    shuffled = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for b, n in enumerate(counts):
        row = table[leader[b]][:shared[b]] if leader[b] != b else []
        take = n - len(row)
        table.append(row + shuffled[at:at + take] + [-1] * (width - n))
        at += take
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    st["k_pages"], st["v_pages"] = normal(P, case["hkv"], S, d), normal(P, case["hkv"], S, d)
    st["table"], st["kv_lens"] = ints(table), ints(kv)
    st["cu_q"], st["max_q"], st["max_kv"] = ints(cu), max(q), max(kv)
    st["decode"] = max(q) == 1
    st["q"] = normal(cu[-1], case["hq"], d)
    if case["op"] == "append_norm":
        st["k"], st["v"] = normal(cu[-1], case["hkv"], d, std=3.0), normal(cu[-1], case["hkv"], d)
        st["q_weight"], st["k_weight"] = normal(d, std=0.2, mean=1.0), normal(d, std=0.2, mean=1.0)
    return st


# ---------------------------------------------------------------- plain forms

def _blocks(case):
    """Blocks of queries, the keys that some of their rows see, and which rows see which: (from, to, keys, mask)."""
    n = case["n"]
    for a in range(0, n, 1024):
        b = min(n, a + 1024)
        lo = _first_key(case, a)
        keys = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, b, device="cuda")])
        row = torch.arange(a, b, device="cuda")[:, None]
        yield a, b, keys, (keys <= row) & ((keys > row - case["window"]) | (keys < case["sinks"]))


def _scores(st, a, b, keys, mask):
    """Scaled scores [B, Hkv, G, rows, keys] of queries a .. b - 1, -inf where a row does not see a key."""
    case, d = st["case"], st["case"]["d"]
    G = case["h"] // case["hkv"]
    q = st["q"][:, :, a:b].float().view(case["b"], case["hkv"], G * (b - a), d)
    s = (q @ st["k"][:, :, keys].float().transpose(-1, -2)).view(case["b"], case["hkv"], G, b - a, len(keys))
    return (s * (1.0 / math.sqrt(d))).masked_fill_(~mask, -math.inf)


def _plain_window(st):
    case, q = st["case"], st["q"]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    for a, b, keys, mask in _blocks(case):
        s = _scores(st, a, b, keys, mask)
        m = s.amax(-1, keepdim=True)   # (every row sees its own key)
        s = s.sub_(m).exp_()
        l = s.sum(-1, keepdim=True)
        x = (s.flatten(2, 3) @ st["v"][:, :, keys].float()).view(*s.shape[:4], case["d"]) / l
        o[:, :, a:b] = x.flatten(1, 2).to(q.dtype)
        lse[:, :, a:b] = (m + l.log()).squeeze(-1).flatten(1, 2)
    return {"o": o, "lse": lse}


def _plain_window_grad(st):
    case, q, k, v = st["case"], st["q"], st["k"], st["v"]
    B, Hkv, G, d = case["b"], case["hkv"], case["h"] // case["hkv"], case["d"]
    scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q)
    dk = torch.zeros(k.shape, dtype=torch.float32, device=k.device)
    dv = torch.zeros_like(dk)
    delta = (st["do"].float() * st["o"].float()).sum(-1)
    for a, b, keys, mask in _blocks(case):
        rows = (B, Hkv, G, b - a)
        s = _scores(st, a, b, keys, mask)
        p = s.sub_(st["lse"][:, :, a:b].view(*rows, 1)).exp_().flatten(2, 3)
        do = st["do"][:, :, a:b].float().view(B, Hkv, -1, d)
        dv[:, :, keys] += p.transpose(-1, -2) @ do
        ds = (do @ v[:, :, keys].float().transpose(-1, -2)).sub_(delta[:, :, a:b].reshape(B, Hkv, -1, 1)).mul_(p)
        dk[:, :, keys] += ds.transpose(-1, -2) @ q[:, :, a:b].float().view(B, Hkv, -1, d) * scale
        dq[:, :, a:b] = (ds @ k[:, :, keys].float() * scale).view(B, case["h"], b - a, d).to(q.dtype)
    return {"dq": dq, "dk": dk.to(k.dtype), "dv": dv.to(v.dtype)}


def _plain_paged(st):
    """Attention over the cache, every sequence padded to the longest; with a window where the case has one."""
    case, table, kv_lens, cu = st["case"], st["table"].long(), st["kv_lens"].long(), st["cu_q"].long()
    q, S, d = st["q"], case["page"], case["d"]
    B, Hkv, G = table.shape[0], case["hkv"], case["hq"] // case["hkv"]
    key = torch.arange(st["max_kv"], device=q.device)
    page = table.clamp(min=0)[:, key // S]
    live = key[None] < kv_lens[:, None]                                               # [B, N]
    k = st["k_pages"][page, :, key % S].float().permute(0, 2, 3, 1)                   # [B, Hkv, d, N]
    v = torch.where(live[:, :, None, None], st["v_pages"][page, :, key % S].float(), 0.0).transpose(1, 2)
    new = torch.arange(st["max_q"], device=q.device)
    n_q = cu[1:] - cu[:-1]
    there = new[None] < n_q[:, None]                                                  # [B, Q]
    token = (cu[:-1, None] + new[None]).clamp(max=q.shape[0] - 1)
    rows = q[token].float().view(B, len(new), Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, d)
    s = (rows @ k).view(B, Hkv, G, len(new), len(key)) * (1.0 / math.sqrt(d))
    position = (kv_lens - n_q)[:, None] + new[None]                                   # [B, Q]
    keep = live[:, None, :] & (key <= position[:, :, None])
    if "window" in case:
        keep = keep & ((key > position[:, :, None] - case["window"]) | (key < case["sinks"]))
    s.masked_fill_(~keep[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    base = torch.where(m == -math.inf, 0.0, m)
    s = s.sub_(base).exp_()
    l = s.sum(-1, keepdim=True)
    o = (s.view(B, Hkv, -1, len(key)) @ v).view(B, Hkv, G, len(new), d) / torch.where(l == 0, 1.0, l)
    lse = (base + l.log()).squeeze(-1)
    out, out_lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    at = token[there]
    out[at] = o.permute(0, 3, 1, 2, 4)[there].reshape(-1, Hkv * G, d).to(q.dtype)
    out_lse[at] = lse.permute(0, 3, 1, 2)[there].reshape(-1, Hkv * G)
    return {"o": out, "lse": out_lse}


def _plain_turn(y, positions, inv_freq, interleaved, sign=1.0):
    """y [..., n, d] fp32 rotated by positions [n]; angles in 64 bits, products in 32."""
    angle = positions.double()[:, None] * inv_freq[None]
    c, s = angle.cos().float(), (angle.sin() * sign).float()
    r, y = 2 * inv_freq.numel(), y.clone()
    if interleaved:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    return y


def _plain_normed(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _plain_norm_rope(st):
    y = _plain_turn(_plain_normed(st["x"], st["weight"]), st["positions"], st["inv_freq"], st["case"]["interleaved"])
    return {"y": y.to(st["x"].dtype)}


def _plain_norm_rope_grad(st):
    x, w = st["x"].float(), st["weight"].float()
    g = _plain_turn(st["dy"].float(), st["positions"], st["inv_freq"], st["case"]["interleaved"], -1.0)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    x = x * r
    dw = (g * x).double().sum((0, 1, 2)).float()   # (a sum over every row)
    g = g * w
    return {"dx": (r * (g - x * (g * x).mean(-1, keepdim=True))).to(st["x"].dtype), "dweight": dw}


def _plain_append_norm(st):
    case, cu, S = st["case"], st["cu_q"].long(), st["case"]["page"]
    token = torch.arange(st["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    pos = st["kv_lens"].long()[seq] - cu[seq + 1] + token

    def turned(x, w):
        y = _plain_turn(_plain_normed(x, w).transpose(0, 1), pos, st["inv_freq"], case["interleaved"])
        return y.transpose(0, 1).to(x.dtype)

    page, slot = st["table"].long()[seq, pos // S], pos % S
    st["k_pages"][page, :, slot] = turned(st["k"], st["k_weight"])
    st["v_pages"][page, :, slot] = st["v"]
    return {"q": turned(st["q"], st["q_weight"]).contiguous(), "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


# ---------------------------------------------------------------- the library's calls

def _own_window(st):
    import exact_attention_17_gb300 as fa2

    o, lse = fa2.forward_window(st["q"], st["k"], st["v"], st["case"]["window"], sinks=st["case"]["sinks"],
                                out_dtype=st["q"].dtype)
    return {"o": o, "lse": lse}


def _own_window_grad(st):
    import exact_attention_17_gb300 as fa2

    dq, dk, dv = fa2.backward_window(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["case"]["window"],
                                     sinks=st["case"]["sinks"], grad_dtype=st["q"].dtype)
    return {"dq": dq, "dk": dk, "dv": dv}


def _own_paged_window(st):
    import exact_attention_17_gb300 as fa2

    o, lse = fa2.forward_paged_window(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                                      st["case"]["window"], sinks=st["case"]["sinks"],
                                      cu_q=None if st["decode"] else st["cu_q"])
    return {"o": o, "lse": lse}


def _own_paged_prefix(st):
    import exact_attention_17_gb300 as fa2

    o, lse = fa2.forward_paged_prefix(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                                      st["cu_groups"], st["prefix_lens"], cu_q=None if st["decode"] else st["cu_q"])
    return {"o": o, "lse": lse}


def _own_norm_rope(st):
    import exact_attention_17_gb300 as fa2

    return {"y": fa2.norm_rope(st["x"], st["weight"], st["positions"], st["inv_freq"], eps=EPS,
                               interleaved=st["case"]["interleaved"])}


def _own_norm_rope_grad(st):
    import exact_attention_17_gb300 as fa2

    dx, dw = fa2.norm_rope_backward(st["dy"], st["x"], st["weight"], st["positions"], st["inv_freq"], eps=EPS,
                                    interleaved=st["case"]["interleaved"])
    return {"dx": dx, "dweight": dw}


def _own_append_norm(st):
    import exact_attention_17_gb300 as fa2

    q = fa2.append_paged(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                         cu_q=None if st["decode"] else st["cu_q"], q=st["q"], inv_freq=st["inv_freq"],
                         interleaved=st["case"]["interleaved"], q_weight=st["q_weight"], k_weight=st["k_weight"],
                         eps=EPS)
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


_PLAIN = {"window": _plain_window, "window_grad": _plain_window_grad, "paged_window": _plain_paged,
          "paged_prefix": _plain_paged, "norm_rope": _plain_norm_rope, "norm_rope_grad": _plain_norm_rope_grad,
          "append_norm": _plain_append_norm}
_OWN = {"window": _own_window, "window_grad": _own_window_grad, "paged_window": _own_paged_window,
        "paged_prefix": _own_paged_prefix, "norm_rope": _own_norm_rope, "norm_rope_grad": _own_norm_rope_grad,
        "append_norm": _own_append_norm}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _seen(position, keys, window, sinks):
    """How many of the first `keys` keys a query at `position` sees."""
    last = min(position, keys - 1)
    lo = max(0, position - window + 1)
    return max(0, last - lo + 1) + min(sinks, lo, last + 1)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    op, d = case["op"], case["d"]
    if op in ("window", "window_grad"):
        b, h, hkv, n = case["b"], case["h"], case["hkv"], case["n"]
        cells = b * h * sum(_seen(i, n, case["window"], case["sinks"]) for i in range(n))
        q, kv, lse = b * h * n * d * size, b * hkv * n * d * size, 4 * b * h * n
        if op == "window":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * cells * d}
        # q, o, do, k, v and the row sums in; dq, dk, dv out; five products
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * cells * d}
    if op in ("norm_rope", "norm_rope_grad"):
        n = case["b"] * case["h"] * case["n"] * d
        small = 4 * case["n"] + 4 * case["rotary"] + size * d
        if op == "norm_rope":
            return {"bytes": 2 * n * size + small, "flops": 4 * n + 3 * n * case["rotary"] // d}
        return {"bytes": 3 * n * size + small + 4 * d, "flops": 11 * n + 3 * n * case["rotary"] // d}
    q, kv = _lengths(case)
    T = sum(q)
    if op == "append_norm":
        turned = T * (case["hq"] + case["hkv"])
        return {"bytes": 2 * T * (case["hq"] + 2 * case["hkv"]) * d * size + 4 * T + 2 * d * size,
                "flops": 4 * turned * d + 3 * turned * case["rotary"]}
    if op == "paged_window":
        cells = keys = 0
        for a, n in zip(q, kv):
            cells += sum(_seen(p, n, case["window"], case["sinks"]) for p in range(n - a, n))
            lo = max(0, n - a - case["window"] + 1)
            keys += n - lo + min(case["sinks"], lo)
    else:
        cells = sum(a * n - a * (a - 1) // 2 for a, n in zip(q, kv))
        first, prefix = _groups(case)
        keys = sum(kv) - sum((first[i + 1] - first[i] - 1) * n for i, n in enumerate(prefix))
    return {"bytes": (2 * T * case["hq"] * d + 2 * keys * case["hkv"] * d) * size + 4 * T * case["hq"]
            + 4 * -(-keys // case["page"]) + 8 * case["seqs"],
            "flops": 4 * cells * case["hq"] * d}


# ---------------------------------------------------------------- the definition in 64 bits

def _turned(x, positions, inv_freq, interleaved, sign=1.0):
    """x [n, ..., d] in 64 bits times the rotation, pair by pair as complex numbers."""
    r = 2 * inv_freq.numel()
    turn = torch.polar(torch.ones_like(inv_freq)[None].expand(len(positions), -1),
                       sign * positions.double()[:, None] * inv_freq[None])
    turn = turn.view(len(positions), *([1] * (x.dim() - 2)), r // 2)
    head = x[..., :r]
    pairs = head.unflatten(-1, (r // 2, 2)) if interleaved else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    out = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    out = out if interleaved else out.transpose(-1, -2)
    return torch.cat([out.flatten(-2), x[..., r:]], -1)


def _normed(x, weight):
    x = x.double()
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.double()


def _exact_window(st):
    """A head and a strip of queries at a time, each strip against all keys up to its last."""
    case, q, d = st["case"], st["q"], st["case"]["d"]
    G, n, grad = case["h"] // case["hkv"], case["n"], st["case"]["op"] == "window_grad"
    shape = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(q.shape, **shape), torch.zeros(q.shape[:3], **shape)
    dq, dk, dv = torch.zeros(q.shape, **shape), torch.zeros(st["k"].shape, **shape), torch.zeros(st["k"].shape, **shape)
    for b in range(case["b"]):
        for h in range(case["h"]):
            k, v = st["k"][b, h // G].double(), st["v"][b, h // G].double()
            for a in range(0, n, 512):
                z = min(n, a + 512)
                lo = max(0, a - case["window"] + 1) // 512 * 512   # (nothing between the sinks and this is seen)
                lo = 0 if lo < case["sinks"] else lo
                j = torch.arange(lo, z, device="cuda")
                if lo > 0 and case["sinks"] > 0:
                    j = torch.cat([torch.arange(case["sinks"], device="cuda"), j])
                i = torch.arange(a, z, device="cuda")[:, None]
                hidden = (j[None] > i) | ((i - j[None] >= case["window"]) & (j[None] >= case["sinks"]))
                x = q[b, h, a:z].double()
                s = torch.einsum("ic,jc->ij", x, k[j]) / math.sqrt(d)
                s[hidden] = -math.inf
                if not grad:
                    lse[b, h, a:z] = torch.logsumexp(s, -1)
                    o[b, h, a:z] = torch.softmax(s, -1) @ v[j]
                    continue
                p = torch.exp(s - st["lse"][b, h, a:z].double()[:, None])
                do = st["do"][b, h, a:z].double()
                ds = p * (torch.einsum("ic,jc->ij", do, v[j]) - (do * st["o"][b, h, a:z].double()).sum(-1)[:, None])
                dq[b, h, a:z] = ds @ k[j] / math.sqrt(d)
                dk[b, h // G].index_add_(0, j, ds.T @ x / math.sqrt(d))
                dv[b, h // G].index_add_(0, j, p.T @ do)
    return {"dq": dq, "dk": dk, "dv": dv} if grad else {"o": o, "lse": lse}


def _exact_paged(st):
    case, S, d = st["case"], st["case"]["page"], st["case"]["d"]
    G = case["hq"] // case["hkv"]
    q_lens, kv_lens = _lengths(case)
    table = st["table"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    out_lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        j = torch.arange(length, device="cuda")
        i = torch.arange(length - n, length, device="cuda")
        hidden = j[None] > i[:, None]
        if "window" in case:
            hidden |= (i[:, None] - j[None] >= case["window"]) & (j[None] >= case["sinks"])
            some = ~hidden.all(0)   # keys that nobody sees are left out
            j, hidden = j[some], hidden[:, some]
        page = torch.tensor(table[b][:-(-length // S)], device="cuda")[j // S]
        for h in range(case["hkv"]):
            k, v = st["k_pages"][page, h, j % S].double(), st["v_pages"][page, h, j % S].double()
            x = st["q"][at:at + n, h * G:(h + 1) * G].double()
            s = torch.einsum("tgc,jc->tgj", x, k) / math.sqrt(d)
            s = s.masked_fill(hidden[:, None], -math.inf)
            out_lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
            out[at:at + n, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
        at += n
    return {"o": out, "lse": out_lse}


def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    op = case["op"]
    if op in ("window", "window_grad"):
        return _exact_window(st)
    if op in ("paged_window", "paged_prefix"):
        return _exact_paged(st)
    if op == "norm_rope":
        y = _turned(_normed(st["x"], st["weight"]).permute(2, 0, 1, 3), st["positions"], st["inv_freq"],
                    case["interleaved"])
        return {"y": y.permute(1, 2, 0, 3).contiguous()}
    if op == "norm_rope_grad":
        g = _turned(st["dy"].double().permute(2, 0, 1, 3), st["positions"], st["inv_freq"], case["interleaved"],
                    -1.0).permute(1, 2, 0, 3)
        x, w = st["x"].double(), st["weight"].double()
        length = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        along = (g * w * x).sum(-1, keepdim=True) / (case["d"] * length ** 3)
        return {"dx": g * w / length - x * along, "dweight": torch.einsum("bhnc,bhnc->c", g, x / length)}
    q_lens, kv_lens = _lengths(case)
    how = (st["inv_freq"], case["interleaved"])
    keys, values = st["k_pages"].double(), st["v_pages"].double()
    table, queries, at = st["table"].tolist(), [], 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        pos = torch.arange(length - n, length, device="cuda")
        page, slot = torch.tensor(table[b], device="cuda")[pos // case["page"]], pos % case["page"]
        queries.append(_turned(_normed(st["q"][at:at + n], st["q_weight"]), pos, *how))
        keys[page, :, slot] = _turned(_normed(st["k"][at:at + n], st["k_weight"]), pos, *how)
        values[page, :, slot] = st["v"][at:at + n].double()
        at += n
    return {"q": torch.cat(queries), "k_pages": keys, "v_pages": values}

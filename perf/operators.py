"""The operators around a paged key/value cache, in plain torch and as the library's calls.

``forward_paged``   attention of a chunk of new tokens (or of one token a sequence) over the cache
``append_paged``    new tokens' keys (rotated) and values into their pages, queries rotated beside them
``rope``            rotary positions and their gradient
``pages``           forking, freeing, reserving, copying and compacting pages

A cache is a pair [P, Hkv, S, d] of key and value pages, a table int32 [B, M] of page numbers (-1:
none) and int32 lengths; sequence b's token t lies in slot t % S of page table[b, t // S].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a short conversation or two: one token each over about a thousand tokens, latency counts
        dict(name="decode_small", op="forward_paged", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=2,
             q_min=1, q_max=1, kv_min=700, kv_max=1000, causal=True, mix=1),
        # a serving batch: one token each, lengths all over the range
        dict(name="decode_batch", op="forward_paged", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=64,
             q_min=1, q_max=1, kv_min=1000, kv_max=8192, causal=True, mix=2),
        # a few very long contexts, small heads
        dict(name="decode_long", op="forward_paged", dtype="fp16", hq=32, hkv=4, d=64, page=64, seqs=4,
             q_min=1, q_max=1, kv_min=100000, kv_max=131072, causal=True, mix=3),
        # a mixed step: chunks of a few to some hundred tokens, an odd number of heads a group
        dict(name="chunk_mixed", op="forward_paged", dtype="bf16", hq=20, hkv=4, d=128, page=32, seqs=12,
             q_min=1, q_max=512, kv_min=600, kv_max=8192, causal=True, mix=4),
        # the second half of a long prompt, heads not shared
        dict(name="chunk_prefill", op="forward_paged", dtype="bf16", hq=32, hkv=32, d=128, page=128, seqs=1,
             q_min=8192, q_max=8192, kv_min=16384, kv_max=16384, causal=True, mix=5),
        # wide heads, every new token sees the whole cache (a cross-attention memory)
        dict(name="chunk_wide", op="forward_paged", dtype="bf16", hq=16, hkv=2, d=256, page=64, seqs=3,
             q_min=100, q_max=1000, kv_min=2000, kv_max=4096, causal=False, mix=6),
        # a decoding step's new tokens
        dict(name="append_step", op="append_paged", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=64,
             q_min=1, q_max=1, kv_min=1000, kv_max=8192, rotary=128, interleaved=False, scaling="none", mix=7),
        # chunks of a prompt, part of the head rotated, interleaved pairs, frequencies stretched
        dict(name="append_chunk", op="append_paged", dtype="fp16", hq=32, hkv=4, d=64, page=64, seqs=5,
             q_min=500, q_max=4096, kv_min=16384, kv_max=131072, rotary=32, interleaved=True, scaling="ramp", mix=8),
        # queries of a training step at the 4096-length configuration, far positions
        dict(name="rope_train", op="rope", dtype="bf16", b=4, h=16, n=4096, d=128, rotary=128,
             interleaved=False, scaling="linear", start=1000000, backward=False, mix=9),
        # the gradient at the 1000-length configuration in 32 bits
        dict(name="rope_grad", op="rope", dtype="fp32", b=2, h=8, n=1000, d=64, rotary=48,
             interleaved=True, scaling="base", start=0, backward=True, mix=10),
        # one step of a beam search: losers freed, winners forked, a token reserved for each
        dict(name="pages_beams", op="pages", kind="beams", dtype="bf16", groups=8, beams=4, planes=8, hkv=8,
             page=16, d=128, pages=2048, kv_min=100, kv_max=500, mix=11),
        # a pool half of whose pages were freed, moved together
        dict(name="pages_compact", op="pages", kind="compact", dtype="bf16", groups=40, beams=1, planes=8, hkv=8,
             page=16, d=128, pages=4096, kv_min=500, kv_max=1000, mix=12),
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
    op = rng.choice(["decode", "chunk", "chunk", "append_paged", "rope", "pages"])
    d = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([16, 16, 32, 64, 128, 256])
    hkv, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    rotary = dict(rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.5,
                  scaling=rng.choice(["none", "linear", "base", "ramp"]))
    if op == "rope":
        b, h, n = _spread(rng, 1, 8), rng.randint(1, 32), _spread(rng, 100, 8192)
        h = max(1, min(h, (1 << 25) // (b * n * d)))
        return dict(op="rope", dtype=rng.choice(["bf16", "fp16", "fp32"]), b=b, h=h, n=n, d=d, **rotary,
                    start=_spread(rng, 1, 1 << 20), backward=rng.random() < 0.5, mix=mix)
    if op == "pages":
        kind = rng.choice(["beams", "compact", "copy"])
        groups, beams = _spread(rng, 2, 32), rng.randint(2, 6) if kind == "beams" else 1
        page = rng.choice([16, 32, 64])
        kv = _range(rng, "kv", 50, 600)
        need = groups * beams * (-(-(kv["kv_max"] + 1) // page) + 1)
        return dict(op="pages", kind=kind, dtype=dtype, groups=groups, beams=beams, planes=rng.choice([2, 4]),
                    hkv=rng.choice([1, 2, 4]), page=page, d=rng.choice([64, 128]),
                    pages=need + rng.randint(1, need), **kv, mix=mix)
    if op == "append_paged":
        case = dict(op=op, dtype=dtype, hq=hkv * group, hkv=hkv, d=d, page=page, seqs=_spread(rng, 1, 64),
                    **_range(rng, "q", 1, 2048), **_range(rng, "kv", 2100, 16384), **rotary, mix=mix)
        while sum(_lengths(case)[0]) * (group + 2) * hkv * d > 1 << 25:
            case["q_min"], case["q_max"] = max(1, case["q_min"] // 2), max(1, case["q_max"] // 2)
    else:
        q = dict(q_min=1, q_max=1) if op == "decode" else _range(rng, "q", 1, 2048)
        case = dict(op="forward_paged", dtype=dtype, hq=hkv * group, hkv=hkv, d=d, page=page,
                    seqs=_spread(rng, 1, 64), **q, **_range(rng, "kv", q["q_max"], 16384),
                    causal=rng.random() < 0.8, mix=mix)
        # the plain form pads every sequence to the longest: bounded in scores and in pages
        while case["seqs"] > 1 and (case["seqs"] * case["hq"] * case["q_max"] * case["kv_max"] > 1 << 31
                                    or case["seqs"] * case["kv_max"] * hkv * d > 1 << 28):
            case["seqs"] = max(1, case["seqs"] // 2)
        if case["hq"] * case["q_max"] * case["kv_max"] > 1 << 31:
            case["hq"] = case["hkv"] * max(1, group // 4)
    return case


def _lengths(case):
    """New tokens and lengths (new tokens among them) of each sequence: (q, kv)."""
    rng = random.Random(case["mix"])
    q = [_spread(rng, case["q_min"], case["q_max"]) for _ in range(case["seqs"])]
    kv = [max(_spread(rng, case["kv_min"], case["kv_max"]), n) for n in q]
    # the ends of the range are met
    q[0] = case["q_max"]
    kv[-1] = max(case["kv_max"], q[-1])
    kv[0] = max(kv[0], q[0])
    return q, kv


def _inv_freq(case):
    """Radians a position of each rotated pair, in 64 bits, with the case's long-context scaling."""
    r, base, factor, length = case["rotary"], 10000.0, 8.0, 4096.0
    if case["scaling"] == "base":
        base *= factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] == "ramp":
        # pairs that turn often within the trained length stay, pairs that turn less than once are stretched
        def pair(turns):
            return r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), r - 1)
        w = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(r // 2)]
        f = [x * (1 - a) + x / factor * a for x, a in zip(f, w)]
    return f


def _mscale(case):
    return 0.1 * math.log(8.0) + 1.0 if case["scaling"] == "ramp" else 1.0


def _beams(case):
    """Page lists of a pool: every group one prompt, its beams sharing the full pages: (rows, lens, refs)."""
    rng = random.Random(case["mix"])
    S, order = case["page"], list(range(case["pages"]))
    rng.shuffle(order)
    if case["kind"] == "beams":
        order.sort(key=lambda p: p >= case["pages"] // 2)   # the upper half is free
    rows, lens, refs, at = [], [], [0] * case["pages"], 0
    for _ in range(case["groups"]):
        n = _spread(rng, case["kv_min"], case["kv_max"])
        full = order[at:at + n // S]
        at += n // S
        for _ in range(case["beams"]):
            row = list(full)
            if n % S:
                row.append(order[at])
                at += 1
            rows.append(row)
            lens.append(n)
            for p in row:
                refs[p] += 1
    return rows, lens, refs


def _losers(case):
    """For each group one beam that is dropped and one that takes its place: (src, dst)."""
    rng = random.Random(case["mix"] + 1)
    src, dst = [], []
    for g in range(case["groups"]):
        a, b = rng.sample(range(case["beams"]), 2)
        src.append(g * case["beams"] + a)
        dst.append(g * case["beams"] + b)
    return src, dst


def _copies(case):
    rng = random.Random(case["mix"] + 2)
    pages = rng.sample(range(case["pages"]), max(2, case["pages"] // 4 * 2))
    half = len(pages) // 2
    return pages[:half], pages[half:2 * half]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dt)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    st = {"case": case}
    if "rotary" in case:
        st["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device="cuda")
        st["mscale"] = _mscale(case)
    if case["op"] == "rope":
        st["x"] = normal(case["b"], case["h"], case["n"], case["d"])
        st["positions"] = torch.arange(case["start"], case["start"] + case["n"], dtype=torch.int32, device="cuda")
        return st
    if case["op"] == "pages":
        rows, lens, refs = _beams(case)
        width = max(-(-(n + 1) // case["page"]) for n in lens) + 1
        flat = [p for row in rows for p in row + [-1] * (width - len(row))]
        B, P = len(rows), case["pages"]
        st["ints0"] = ints(flat + lens + refs)
        st["ints"] = st["ints0"].clone()
        st["table"] = st["ints"][:B * width].view(B, width)
        st["lens"] = st["ints"][B * width:B * width + B]
        st["refs"] = st["ints"][B * width + B:]
        st["pools"] = normal(case["planes"], P, case["hkv"], case["page"], case["d"])
        if case["kind"] == "beams":
            src, dst = _losers(case)
            st["src"], st["dst"], st["add"] = ints(src), ints(dst), ints([1] * B)
        if case["kind"] == "copy":
            src, dst = _copies(case)
            st["src"], st["dst"] = ints(src), ints(dst)
        return st
    # a cache whose pages lie in no order, some of them nobody's
    q, kv = _lengths(case)
    S = case["page"]
    counts = [-(-n // S) for n in kv]
    P, width = sum(counts) + max(4, sum(counts) // 16), max(counts)
    shuffled = torch.randperm(P, generator=torch.Generator().manual_seed(seed)).tolist()
    table, at = [], 0
    for n in counts:
        table.append(shuffled[at:at + n] + [-1] * (width - n))
        at += n
    cu = [0]
    for n in q:
        cu.append(cu[-1] + n)
    st["k_pages"], st["v_pages"] = normal(P, case["hkv"], S, case["d"]), normal(P, case["hkv"], S, case["d"])
    st["table"], st["kv_lens"] = ints(table), ints(kv)
    st["cu_q"], st["max_q"], st["max_kv"] = ints(cu), max(q), max(kv)
    st["decode"] = max(q) == 1
    st["q"] = normal(cu[-1], case["hq"], case["d"])
    if case["op"] == "append_paged":
        st["k"], st["v"] = normal(cu[-1], case["hkv"], case["d"]), normal(cu[-1], case["hkv"], case["d"])
    return st


# ---------------------------------------------------------------- plain forms

def _plain_forward_paged(st):
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
    keep = live[:, None, :]
    if case["causal"]:
        keep = keep & (key[None, None] <= (kv_lens - n_q)[:, None, None] + new[None, :, None])
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


def _plain_rotate(x, positions, inv_freq, interleaved, mscale, sign=1.0):
    """x [..., n, d] rotated by positions [n]; angles in 64 bits, products in 32."""
    angle = positions.double()[:, None] * inv_freq[None]
    c, s = (angle.cos() * mscale).float(), (angle.sin() * (mscale * sign)).float()
    r = 2 * inv_freq.numel()
    y = x.float()
    y = y.clone() if y.data_ptr() == x.data_ptr() else y
    if interleaved:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    return y.to(x.dtype)


def _plain_append_paged(st):
    case, cu, S = st["case"], st["cu_q"].long(), st["case"]["page"]
    token = torch.arange(st["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu, token, right=True) - 1
    pos = st["kv_lens"].long()[seq] - cu[seq + 1] + token
    how = (pos, st["inv_freq"], case["interleaved"], st["mscale"])
    page, slot = st["table"].long()[seq, pos // S], pos % S
    st["k_pages"][page, :, slot] = _plain_rotate(st["k"].transpose(0, 1), *how).transpose(0, 1)
    st["v_pages"][page, :, slot] = st["v"]
    return {"q": _plain_rotate(st["q"].transpose(0, 1), *how).transpose(0, 1).contiguous(),
            "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_rope(st):
    case = st["case"]
    return _plain_rotate(st["x"], st["positions"], st["inv_freq"], case["interleaved"], st["mscale"],
                         -1.0 if case["backward"] else 1.0)


def _plain_free(table, lens, refs, seqs):
    rows = table[seqs]
    refs.index_add_(0, rows[rows >= 0], torch.full_like(rows[rows >= 0], -1, dtype=torch.int32))
    table[seqs] = -1
    lens[seqs] = 0


def _plain_fork(table, lens, refs, src, dst, pools, S):
    rows, n_full, part = table[src].long(), (lens[src] // S).long(), lens[src] % S > 0
    full = torch.arange(table.shape[1], device=table.device)[None] < n_full[:, None]
    shared = rows[full]
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    fresh = (refs == 0).nonzero().flatten()[:int(part.sum())]
    table[dst] = torch.where(full, rows, -1).int()
    table[dst[part], n_full[part]] = fresh.int()
    refs[fresh] = 1
    lens[dst] = lens[src]
    pools[:, fresh] = pools[:, rows[part, n_full[part]]]


def _plain_reserve(table, lens, refs, add, S):
    have, want = (lens + S - 1) // S, (lens + add + S - 1) // S
    grow = (want - have).long()
    seq = torch.repeat_interleave(torch.arange(len(lens), device=lens.device), grow)
    fresh = (refs == 0).nonzero().flatten()[:len(seq)]
    first = grow.cumsum(0) - grow
    slot = have[seq].long() + torch.arange(len(seq), device=lens.device) - first[seq]
    table[seq, slot] = fresh.int()
    refs[fresh] = 1
    lens += add


def _plain_compact(table, refs, pools):
    used = refs > 0
    count = used.sum()
    index = torch.arange(len(refs), device=refs.device)
    movers, holes = index[used & (index >= count)], index[~used & (index < count)]
    moved = torch.where(used, index, -1)
    moved[movers] = holes
    pools[:, holes] = pools[:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, moved[table.clamp(min=0).long()].int(), -1))
    return moved.int()


def _plain_pages(st):
    case, table, lens, refs, pools = st["case"], st["table"], st["lens"], st["refs"], st["pools"]
    st["ints"].copy_(st["ints0"])   # every pass starts from the same tables
    out = {"table": table, "lens": lens, "refs": refs, "pools": pools}
    if case["kind"] == "beams":
        _plain_free(table, lens, refs, st["dst"].long())
        _plain_fork(table, lens, refs, st["src"].long(), st["dst"].long(), pools, case["page"])
        _plain_reserve(table, lens, refs, st["add"], case["page"])
    elif case["kind"] == "compact":
        out["moved"] = _plain_compact(table, refs, pools)
    else:
        pools[:, st["dst"].long()] = pools[:, st["src"].long()]
    return out


# ---------------------------------------------------------------- the library's calls

def _own_forward_paged(st):
    import exact_attention_17_gb300 as fa2

    o, lse = fa2.forward_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                               cu_q=None if st["decode"] else st["cu_q"], causal=st["case"]["causal"])
    return {"o": o, "lse": lse}


def _own_append_paged(st):
    import exact_attention_17_gb300 as fa2

    q = fa2.append_paged(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                         cu_q=None if st["decode"] else st["cu_q"], q=st["q"], inv_freq=st["inv_freq"],
                         interleaved=st["case"]["interleaved"], mscale=st["mscale"])
    return {"q": q, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _own_rope(st):
    import exact_attention_17_gb300 as fa2

    call = fa2.rope_backward if st["case"]["backward"] else fa2.rope
    return call(st["x"], st["positions"], st["inv_freq"], interleaved=st["case"]["interleaved"],
                mscale=st["mscale"])


def _own_pages(st):
    import exact_attention_17_gb300 as fa2

    case, table, lens, refs, pools = st["case"], st["table"], st["lens"], st["refs"], st["pools"]
    st["ints"].copy_(st["ints0"])
    out = {"table": table, "lens": lens, "refs": refs, "pools": pools}
    if case["kind"] == "beams":
        fa2.pages_free(table, lens, refs, st["dst"])
        fa2.pages_fork(table, lens, refs, st["src"], st["dst"], pools)
        fa2.pages_reserve(table, lens, refs, st["add"], case["page"])
    elif case["kind"] == "compact":
        out["moved"] = fa2.pages_compact(table, lens, refs, pools)
    else:
        fa2.pages_copy(pools, st["src"], st["dst"])
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"forward_paged": _own_forward_paged, "append_paged": _own_append_paged, "rope": _own_rope,
                "pages": _own_pages}[op](state)
    return {"forward_paged": _plain_forward_paged, "append_paged": _plain_append_paged, "rope": _plain_rope,
            "pages": _plain_pages}[op](state)


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "rope":
        n = case["b"] * case["h"] * case["n"] * case["d"]
        return {"bytes": 2 * n * size + 4 * case["n"] + 4 * case["rotary"],
                "flops": 3 * n * case["rotary"] // case["d"]}
    if case["op"] == "pages":
        page = case["planes"] * case["hkv"] * case["page"] * case["d"] * size
        rows, lens, refs = _beams(case)
        small = 4 * (len(refs) + sum(len(r) for r in rows) + len(lens))
        if case["kind"] == "beams":
            copies = sum(lens[s] % case["page"] > 0 for s in _losers(case)[0])
        elif case["kind"] == "compact":
            count = sum(r > 0 for r in refs)
            copies = sum(r > 0 for r in refs[count:])
        else:
            copies, small = len(_copies(case)[0]), 0
        return {"bytes": 2 * copies * page + 2 * small, "flops": 0}
    q, kv = _lengths(case)
    if case["op"] == "append_paged":
        n = sum(q) * (case["hq"] + 2 * case["hkv"]) * case["d"]
        rotated = sum(q) * (case["hq"] + case["hkv"]) * case["rotary"]
        return {"bytes": 2 * n * size + 4 * sum(q), "flops": 3 * rotated}
    cells = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(q, kv))
    pages = sum(-(-n // case["page"]) for n in kv)
    return {"bytes": (2 * sum(q) * case["hq"] * case["d"] + 2 * sum(kv) * case["hkv"] * case["d"]) * size
            + 4 * sum(q) * case["hq"] + 4 * pages + 8 * case["seqs"],
            "flops": 4 * cells * case["hq"] * case["d"]}


# ---------------------------------------------------------------- the definition in 64 bits

def _turned(x, positions, inv_freq, interleaved, mscale, sign):
    """x [n, ..., d] in 64 bits times the rotation, pair by pair as complex numbers."""
    r = 2 * inv_freq.numel()
    turn = torch.polar(torch.full_like(inv_freq, mscale)[None].expand(len(positions), -1),
                       sign * positions.double()[:, None] * inv_freq[None])
    turn = turn.view(len(positions), *([1] * (x.dim() - 2)), r // 2)
    head = x[..., :r].double()
    pairs = head.unflatten(-1, (r // 2, 2)) if interleaved else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    out = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    out = out if interleaved else out.transpose(-1, -2)
    return torch.cat([out.flatten(-2), x[..., r:].double()], -1)


def exact(case, seed):
    if case["op"] == "pages":
        return None
    st = prepare(case, seed)
    if case["op"] == "rope":
        y = _turned(st["x"].permute(2, 0, 1, 3), st["positions"], st["inv_freq"], case["interleaved"],
                    st["mscale"], -1.0 if case["backward"] else 1.0)
        return y.permute(1, 2, 0, 3).contiguous()
    q_lens, kv_lens = _lengths(case)
    S, d, G = case["page"], case["d"], case["hq"] // case["hkv"]
    table = st["table"].tolist()
    if case["op"] == "append_paged":
        how = (st["inv_freq"], case["interleaved"], st["mscale"], 1.0)
        keys, values = st["k_pages"].double(), st["v_pages"].double()
        queries, at = [], 0
        for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
            pos = torch.arange(length - n, length, device="cuda")
            queries.append(_turned(st["q"][at:at + n], pos, *how))
            page = torch.tensor(table[b], device="cuda")[pos // S]
            keys[page, :, pos % S] = _turned(st["k"][at:at + n], pos, *how)
            values[page, :, pos % S] = st["v"][at:at + n].double()
            at += n
        return {"q": torch.cat(queries), "k_pages": keys, "v_pages": values}
    if work(case)["flops"] > 4e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    out_lse = torch.full(st["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, length) in enumerate(zip(q_lens, kv_lens)):
        pages = torch.tensor(table[b][:-(-length // S)], device="cuda")
        pos = torch.arange(length, device="cuda")
        for h in range(case["hkv"]):
            k = st["k_pages"][pages, h].reshape(-1, d)[:length].double()
            v = st["v_pages"][pages, h].reshape(-1, d)[:length].double()
            for first in range(0, n, 2048):
                last = min(n, first + 2048)
                x = st["q"][at + first:at + last, h * G:(h + 1) * G].double()
                s = torch.einsum("tgc,jc->tgj", x, k) / math.sqrt(d)
                if case["causal"]:
                    row = torch.arange(first, last, device="cuda") + (length - n)
                    s = s.masked_fill((pos[None] > row[:, None])[:, None], -math.inf)
                z = torch.logsumexp(s, -1)
                out_lse[at + first:at + last, h * G:(h + 1) * G] = z
                out[at + first:at + last, h * G:(h + 1) * G] = torch.exp(s - z[..., None]) @ v
        at += n
    return {"o": out, "lse": out_lse}

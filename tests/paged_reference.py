"""Plain 64-bit forms of the paged-cache operators, and caches to run them on.

Not a test module: the GPU tests import it.  The caches hold NaN in every slot
that belongs to nobody (unused pages, slots behind a sequence's last token), and
their tables hold numbers far outside the pool behind each row's last page.
"""
import gc
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step


class Cache:
    def __init__(self, kv, Hkv, S, d, dtype, seed=0, layout="phsd", spare=3, std=1.0):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.S = list(kv), S
        counts = [-(-n // S) for n in kv]
        P = sum(counts) + spare
        shape = (P, Hkv, S, d) if layout != "pshd" else (P, S, Hkv, d)
        if layout == "layers":     # one layer of a larger pool, K and V of a page next to each other
            pool = torch.full((P, 3, 2, Hkv, S, d), float("nan"), dtype=dtype, device="cuda")
            self.k, self.v = pool[:, 1, 0], pool[:, 1, 1]
        else:
            self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(2))
            if layout == "pshd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = torch.randperm(P, generator=g).tolist()
        width = max([1] + counts)
        self.table = torch.full((len(kv), width), 1 << 30, dtype=torch.int32)
        self.keys, self.values = [], []
        for b, n in enumerate(kv):
            pages, order = order[:counts[b]], order[counts[b]:]
            self.table[b, :counts[b]] = torch.tensor(pages, dtype=torch.int32)
            k = (torch.randn(n, Hkv, d, generator=g) * std).to(dtype).cuda()
            v = torch.randn(n, Hkv, d, generator=g).to(dtype).cuda()
            pos = torch.arange(n, device="cuda")
            page = torch.tensor(pages, dtype=torch.long, device="cuda")[pos // S]
            self.k[page, :, pos % S] = k
            self.v[page, :, pos % S] = v
            self.keys.append(k)
            self.values.append(v)
        self.table = self.table.cuda()
        self.lens = torch.tensor(kv, dtype=torch.int32, device="cuda")


def offsets(q_lens):
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def attention(q, keys, values, q_lens, causal, scale, dtype, out_eps):
    """(O, LSE, bound of |dO|, bound of |dLSE|) in 64 bits.

    First-order bounds.  With u half a step of the input type, A = sum_j p_j
    |v_j|: rounding each P to that type costs at most u A, rounding O out_eps
    |O|.  A score is a sum of d products in fp32: its error is at most delta = 2
    d 2^-24 scale max_j sum_c |q_c k_jc| (2: the tensor core may truncate), which
    changes every weight by at most a relative 2 delta after normalisation; the
    exponential (2^-21) and the row sum (n 2^-24) add to that.  fp16 P below
    2^-14 are rounded with an absolute error of at most 2^-25 while the row's
    largest P is at least 1.
    """
    O, L, bO, bL = [], [], [], []
    at, u = 0, EPS[dtype]
    Hq, d = q.shape[1], q.shape[2]
    for b, n in enumerate(q_lens):
        x = q[at:at + n].double()
        at += n
        k, v = keys[b].double(), values[b].double()
        G = Hq // k.shape[1]
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        s = torch.einsum("thd,jhd->thj", x, k) * scale
        m = k.shape[0]
        keep = torch.ones(n, m, dtype=torch.bool, device=q.device)
        if causal:
            keep = torch.arange(m, device=q.device)[None] <= (torch.arange(n, device=q.device) + m - n)[:, None]
        s = s.masked_fill(~keep[:, None], -math.inf)
        lse = torch.logsumexp(s, -1) if m else torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
        p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
        o = torch.einsum("thj,jhd->thd", p, v)
        A = torch.einsum("thj,jhd->thd", p, v.abs())
        delta = torch.zeros(n, Hq, dtype=torch.float64, device=q.device)
        if m:
            mag = torch.einsum("thd,jhd->thj", x.abs(), k.abs()).masked_fill(~keep[:, None], 0.0)
            delta = 2 * d * 2.0 ** -24 * scale * mag.amax(-1)
        rel = 2 * (delta + 2.0 ** -21 + m * 2.0 ** -24)
        tiny = 2.0 ** -25 * torch.einsum("tj,jhd->thd", keep.double(), v.abs()) if dtype is torch.float16 else 0.0
        O.append(o)
        L.append(lse)
        bO.append((u + rel[..., None]) * A + out_eps * o.abs() + tiny + 1e-30)
        bL.append(rel + lse.abs().nan_to_num(0.0, posinf=0.0) * 2.0 ** -22 + 2.0 ** -22)
    cat = lambda t, shape: torch.cat(t) if t else torch.zeros(shape, dtype=torch.float64, device=q.device)  # noqa: E731
    return cat(O, (0, Hq, d)), cat(L, (0, Hq)), cat(bO, (0, Hq, d)), cat(bL, (0, Hq))


def rotate(x, positions, inv_freq, interleaved, mscale=1.0, sign=1.0):
    """x [..., n, d] in 64 bits, positions [n]."""
    r = 2 * inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq.double()[None]
    c, s = angle.cos() * mscale, angle.sin() * mscale * sign
    y = x.double().clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    a, b = a.clone(), b.clone()
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, b * c + a * s
    return y


def rotate_bound(x, inv_freq, interleaved, dtype, mscale=1.0):
    """|error| of a rotated row: both products of a pair, each of (|a| + |b|) m,
    carry the angle's error (2 pi 2^-25 turns, and 2^-22 for sincospif and the fp32
    products), and the result is rounded once to the type (fp16: subnormals to
    2^-25)."""
    r = 2 * inv_freq.numel()
    y = x.double().abs().clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    both = (a + b) * abs(mscale)
    out = torch.zeros_like(y)
    bound = both * (EPS[dtype] * (1 + 2.0 ** -20) + 2 * math.pi * 2.0 ** -25 + 2.0 ** -22) + 2.0 ** -25
    if interleaved:
        out[..., 0:r:2], out[..., 1:r:2] = bound, bound
    else:
        out[..., :r // 2], out[..., r // 2:r] = bound, bound
    return out


def release_memory():
    """Leaves the device's memory to the next test module as it was found: what
    exceptions' frames hold, the workspaces of matrix products, cached blocks."""
    gc.collect()
    torch.cuda.synchronize()
    torch._C._cuda_clearCublasWorkspaces()
    torch.cuda.empty_cache()

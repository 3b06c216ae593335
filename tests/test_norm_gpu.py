"""Heads normed and rotated in one pass, alone and on the way into a paged cache, and their gradients."""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, Cache, offsets, release_memory, rotate

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    libbuild.build()
    fa2.fa2_device_status(None, reset=True)
    yield
    assert fa2.fa2_device_status(None, reset=True) == fa2.FA2_OK
    release_memory()


def normal(shape, dtype, seed, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std + mean).to(dtype).cuda()


def close(y, ref, bound):
    worst = ((y.double() - ref).abs() / (bound + 1e-30)).max() if y.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.3f} of the bound"


def both(a, freq, interleaved, mscale):
    """|a| + |partner| of rotated columns times mscale, |a| of the others."""
    r, y = 2 * freq.numel(), a.double().abs().clone()
    x0, x1 = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    s = (x0 + x1) * abs(mscale)
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = s, s.clone()
    else:
        y[..., :r // 2], y[..., r // 2:r] = s, s.clone()
    return y


# fp32 errors, relative to the sizes they arise at: an angle (2 pi 2^-25, and 2^-22 for its sine), rsqrtf (2 steps,
# 2^-22), a sum of d positive squares (d 2^-24, halved by the root), and a handful of products (2^-24 each).
def slack(d):
    return 2 * math.pi * 2.0 ** -25 + 2.0 ** -22 + 2.0 ** -22 + d * 2.0 ** -25 + 8 * 2.0 ** -24


def forward_64(x, w, pos, freq, eps, interleaved, mscale):
    """x [..., n, d] -> (y, bound)"""
    x, w = x.double(), w.double()
    u = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    y = rotate(u, pos, freq, interleaved, mscale)
    return y, both(u, freq, interleaved, mscale) * slack(x.shape[-1]), y.abs()


def backward_64(dy, x, w, pos, freq, eps, interleaved, mscale, chain):
    d = x.shape[-1]
    x, w = x.double(), w.double()
    g = rotate(dy, pos, freq, interleaved, mscale, -1.0)
    big = both(dy, freq, interleaved, mscale)                 # what g's errors are relative to
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    dx = r * (g * w - x * r * r * (g * w * x).sum(-1, keepdim=True) / d)
    size = (big * w.abs() * x.abs()).sum(-1, keepdim=True)
    # the sum of d products (d 2^-24) and three powers of r
    bound = (slack(d) * 4 + d * 2.0 ** -24) * (r * big * w.abs() + x.abs() * r ** 3 * size / d)
    rows = tuple(range(x.dim() - 1))
    dw = (g * x * r).sum(rows)
    dw_bound = (slack(d) * 2 + chain * 2.0 ** -24) * (big * x.abs() * r).sum(rows)
    return dx, bound, dw, dw_bound


def rounded(bound, y, dtype):
    """...and one rounding to the type (fp16: subnormals to 2^-25)."""
    return bound * (1 + 2 * EPS[dtype]) + EPS[dtype] * y.abs() + 2.0 ** -25


CASES = [
    # dtype, B, H, N, d, rotary, interleaved, first position, fp32 weights
    (BF, 1, 1, 1, 64, 64, False, 0, False),
    (BF, 2, 3, 5, 128, 128, False, 7, True),
    (HF, 1, 8, 100, 128, 64, True, 1000, False),
    (F32, 2, 2, 33, 64, 48, True, 0, True),
    (F32, 2, 2, 33, 64, 48, False, 131071, True),
    (BF, 1, 40, 17, 256, 256, True, 1 << 20, False),
    (BF, 3, 5, 300, 128, 96, False, (1 << 31) - 400, True),
    (HF, 1, 2, 9, 64, 20, False, 3, False),         # halves that fill no vector
    (BF, 2, 2, 9, 128, 20, True, 3, True),
    (F32, 1, 3, 21, 256, 34, False, 11, True),
    (F32, 1, 3, 21, 256, 256, True, 11, True),
    (BF, 1, 9, 4000, 64, 64, False, 100000, False),
    (HF, 1, 2, 50, 256, 0, False, -20, True),       # no rotation
    (BF, 1, 2, 50, 128, 128, True, -20, False),     # positions below zero
    (F32, 5, 7, 1001, 128, 128, False, 5, True),
]
IDS = [f"{str(c[0])[6:]}-{c[1]}x{c[2]}x{c[3]}x{c[4]}-r{c[5]}{'i' if c[6] else 'h'}" for c in CASES]


def arguments(case):
    dtype, B, H, N, d, r, interleaved, start, wide = case
    x = normal((B, H, N, d), dtype, seed=N) * normal((B, H, N, 1), dtype, seed=1, std=0.5).exp()
    w = normal((d,), F32 if wide else dtype, seed=2, std=0.3, mean=1.0)
    freq = fa2.rope_inv_freq(r, device="cuda") if r else torch.zeros(0, dtype=torch.float64, device="cuda")
    pos = torch.arange(start, start + N, dtype=torch.int64 if start % 2 else torch.int32, device="cuda")
    return x, w, freq, pos, dict(eps=1e-5, interleaved=interleaved, mscale=1.25)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_matches_the_64_bit_form(case):
    x, w, freq, pos, how = arguments(case)
    y = fa2.norm_rope(x, w, pos, freq if freq.numel() else None, **how)
    ref, bound, size = forward_64(x, w, pos, freq, **how)
    close(y, ref, rounded(bound, size, x.dtype))
    z = x.clone()
    assert fa2.norm_rope(z, w, pos, freq, **how, out=z) is z
    assert torch.equal(z, y)


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_gradients_match_the_64_bit_form(case):
    x, w, freq, pos, how = arguments(case)
    B, H, N, d = x.shape
    dy = normal(x.shape, x.dtype, seed=3)
    dx, dw = fa2.norm_rope_backward(dy, x, w, pos, freq, **how)
    # a lane adds up the rows it sees one after the other (all heads of its tokens: tiles of at most 8 tokens and 304
    # blocks at least 128 of them running at the same time), then trees and 32 strips of the blocks
    chain = H * -(-B * N // (8 * 128)) + 128
    ref, bound, ref_w, bound_w = backward_64(dy, x, w, pos, freq, **how, chain=chain)
    close(dx, ref, rounded(bound, ref, x.dtype))
    assert dw.dtype is F32
    close(dw, ref_w, bound_w)
    # in place, over either, and the same bits again
    for other in (dy, x):
        z = other.clone()
        args = (z, x) if other is dy else (dy, z)
        dx2, dw2 = fa2.norm_rope_backward(*args, w, pos, freq, **how, dx=z)
        assert dx2 is z and torch.equal(z, dx) and torch.equal(dw2, dw)


def test_gradients_against_differences():
    """Central differences of sum(c * y) in 64 bits, of the 64-bit form: step^2 terms of 1e-8 and rounding of fp32."""
    d, how = 64, dict(eps=1e-3, interleaved=False, mscale=1.5)
    x, c, w = normal((1, 2, 3, d), F32, 4), normal((1, 2, 3, d), F32, 5), normal((d,), F32, 6, 0.3, 1.0)
    freq, pos = fa2.rope_inv_freq(32, device="cuda"), torch.tensor([5, 90, 4096], dtype=torch.int32, device="cuda")
    f = lambda a, b: (c.double() * forward_64(a, b, pos, freq, **how)[0]).sum().item()  # noqa: E731
    dx, dw = fa2.norm_rope_backward(c, x, w, pos, freq, **how)
    h = 1e-4
    for e in range(0, x.numel(), 11):
        step = torch.zeros(x.numel(), dtype=torch.float64, device="cuda")
        step[e] = h
        step = step.view(x.shape)
        assert abs((f(x + step, w) - f(x - step, w)) / (2 * h) - dx.view(-1)[e].item()) < 2e-5
    for e in range(0, d, 5):
        step = torch.zeros(d, dtype=torch.float64, device="cuda")
        step[e] = h
        assert abs((f(x, w + step) - f(x, w - step)) / (2 * h) - dw[e].item()) < 2e-5


def test_packed_tokens_strides_and_batched_positions():
    T, H, d = 77, 6, 128
    how = dict(eps=1e-6, interleaved=False, mscale=1.0)
    freq, w = fa2.rope_inv_freq(64, device="cuda"), normal((d,), BF, 9, 0.3, 1.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    for columns in (d + 8, d + 3):   # rows on 16-byte boundaries, and off them
        x = normal((T, 3, H, columns), BF, seed=1)[:, 1, :, :d]
        ref, bound, size = forward_64(x.transpose(0, 1), w, pos, freq, **how)
        bound = rounded(bound, size, BF)
        close(fa2.norm_rope(x, w, pos, freq).transpose(0, 1), ref, bound)
        out = torch.empty((H, T, d), dtype=BF, device="cuda").transpose(0, 1)
        close(fa2.norm_rope(x, w, pos, freq, out=out).transpose(0, 1), ref, bound)
        dy = normal((T, H, columns), BF, seed=3)[..., :d]
        dx, dw = fa2.norm_rope_backward(dy, x, w, pos, freq)
        rx, bx, rw, bw = backward_64(dy.transpose(0, 1), x.transpose(0, 1), w, pos, freq, **how, chain=200)
        close(dx.transpose(0, 1), rx, rounded(bx, rx, BF))
        close(dw, rw, bw)
    # positions of their own for each batch; a batch read twice, gradients of one row for all heads
    x = normal((1, H, 30, d), BF, seed=3).expand(2, H, 30, d)
    dy = normal((2, 1, 30, d), BF, seed=4).expand(2, H, 30, d)
    pos = torch.stack([torch.arange(30), torch.arange(30) * 1000]).cuda()
    y = fa2.norm_rope(x, w, pos, freq, interleaved=True)
    dx, dw = fa2.norm_rope_backward(dy, x, w, pos, freq, interleaved=True)
    how["interleaved"] = True
    total, slacks = 0.0, 0.0
    for b in range(2):
        ref, bound, size = forward_64(x[b], w, pos[b], freq, **how)
        close(y[b], ref, rounded(bound, size, BF))
        rx, bx, rw, bw = backward_64(dy[b], x[b], w, pos[b], freq, **how, chain=200)
        close(dx[b], rx, rounded(bx, rx, BF))
        total, slacks = total + rw, slacks + bw
    close(dw, total, slacks)


def test_rows_of_zeros_and_no_rows():
    w, freq = normal((64,), BF, 1), fa2.rope_inv_freq(64, device="cuda")
    pos = torch.arange(4, device="cuda")
    x = torch.zeros((1, 2, 4, 64), dtype=BF, device="cuda")
    dy = normal(x.shape, BF, 2)
    assert not fa2.norm_rope(x, w, pos, freq).any()
    dx, dw = fa2.norm_rope_backward(dy, x, w, pos, freq, eps=1e-6)
    assert not dw.any()
    ref, bound, _, _ = backward_64(dy, x, w, pos, freq, 1e-6, False, 1.0, 1)
    close(dx, ref, rounded(bound, ref, BF))
    for shape in ((0, 2, 4, 64), (1, 0, 4, 64), (1, 2, 0, 64)):
        x = torch.zeros(shape, dtype=BF, device="cuda")
        pos = torch.arange(shape[2], device="cuda")
        assert fa2.norm_rope(x, w, pos, freq).shape == shape
        dx, dw = fa2.norm_rope_backward(x, x, w, pos, freq, dweight=torch.full((64,), 7.0, device="cuda"))
        assert dx.shape == shape and not dw.any()


APPEND = [
    # dtype, d, Hq, Hkv, page, q lengths, lengths, rotary, interleaved, weights
    (BF, 128, 8, 2, 16, [1, 1, 1], [1, 16, 17], 128, False, "both"),
    (HF, 64, 4, 4, 32, [5, 0, 40, 1], [5, 3, 100, 33], 32, True, "fp32"),
    (BF, 256, 6, 2, 64, [130, 7], [400, 7], 64, False, "q"),
    (BF, 128, 0, 3, 128, [9, 300], [9, 1000], 0, False, "k"),
    (HF, 128, 16, 1, 1024, [20, 3], [1500, 2000], 20, False, "both"),     # halves that fill no vector
    (BF, 64, 3, 3, 16, [10, 20], [4, 20], 64, True, "k"),                # more new tokens than the length
    (BF, 128, 32, 8, 16, [1] * 70, [(31 * i) % 500 + 1 for i in range(70)], 128, False, "fp32"),
]


@pytest.mark.parametrize("layout", ["phsd", "pshd", "layers"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{str(c[0])[6:]}-d{c[1]}-h{c[2]}.{c[3]}-s{c[4]}-r{c[7]}-{c[9]}")
def test_append_writes_the_new_tokens_alone(case, layout):
    dtype, d, Hq, Hkv, S, q_lens, kv, r, interleaved, weights = case
    cache = Cache(kv, Hkv, S, d, dtype, seed=5, layout=layout)
    T = sum(q_lens)
    k, v = normal((T + 3, Hkv, d), dtype, 6), normal((T + 3, Hkv, d), dtype, 7)
    q = normal((T + 3, Hq, d), dtype, 8) if Hq else None
    freq = fa2.rope_inv_freq(r, device="cuda") if r else None
    kind = F32 if weights == "fp32" else dtype
    qw = None if weights == "k" else normal((d,), kind, 9, 0.3, 1.0)
    kw = None if weights == "q" else normal((d,), kind, 10, 0.3, 1.0)
    before_k, before_v = cache.k.clone(), cache.v.clone()
    q_out = None if q is None else torch.full_like(q, 7.0)
    how = dict(interleaved=interleaved, mscale=1.25)
    got = fa2.append_paged(k, v, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens), q=q, q_out=q_out,
                           inv_freq=freq, q_weight=qw, k_weight=kw, eps=1e-5, **how)
    assert got is q_out
    freq = torch.zeros(0, dtype=torch.float64, device="cuda") if freq is None else freq

    def check(y, x, w, pos):
        x, pos = x.transpose(0, 1), pos
        if w is None:
            ref = rotate(x, pos, freq, **how)
            bound, size = both(x, freq, interleaved, 1.25) * slack(d), ref.abs()
        else:
            ref, bound, size = forward_64(x, w, pos, freq, 1e-5, **how)
        close(y.transpose(0, 1), ref, rounded(bound, size, dtype))

    at = 0
    for b, (n, length) in enumerate(zip(q_lens, kv)):
        pos = torch.arange(length - n, length, device="cuda")
        rows = slice(at, at + n)
        at += n
        if q is not None:
            check(q_out[rows], q[rows], qw, pos)
        there = pos >= 0
        pos, new_k, new_v = pos[there], k[rows][there], v[rows][there]
        page, slot = cache.table[b].long()[pos // S], pos % S
        check(cache.k[page, :, slot], new_k, kw, pos)
        assert torch.equal(cache.v[page, :, slot], new_v)
        before_k[page, :, slot] = cache.k[page, :, slot]
        before_v[page, :, slot] = new_v
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    assert same(cache.k, before_k) and same(cache.v, before_v)
    assert q_out is None or (q_out[T:] == 7.0).all()


def test_a_step_with_normed_heads_is_captured_and_replayed():
    """Room, append and attention of single tokens, captured once and replayed with longer sequences."""
    d, Hq, Hkv, S, B = 128, 8, 2, 16, 3
    pool = torch.zeros((2, 40, Hkv, S, d), dtype=BF, device="cuda")
    table = torch.full((B, 8), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, 40))
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    freq = fa2.rope_inv_freq(d, device="cuda")
    qw, kw = normal((d,), F32, 1, 0.3, 1.0), normal((d,), F32, 2, 0.3, 1.0)
    steps = 21
    q, k, v = normal((steps, B, Hq, d), BF, 3), normal((steps, B, Hkv, d), BF, 4), normal((steps, B, Hkv, d), BF, 5)
    now = [t[0].clone() for t in (q, k, v)]

    def step():
        fa2.pages_reserve(table, lens, refs, one, S)
        rq = fa2.append_paged(now[1], now[2], pool[0], pool[1], table, lens, q=now[0], inv_freq=freq, q_weight=qw,
                              k_weight=kw)
        return fa2.forward_paged(rq, pool[0], pool[1], table, lens)[0]

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()                                     # (a warm-up, taken back)
        for t, value in ((table, -1), (lens, 0), (refs, 0)):
            t.fill_(value)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step()
    got = []
    for i in range(steps):
        for t, src in zip(now, (q, k, v)):
            t.copy_(src[i])
        graph.replay()
        got.append(out.clone())
    got = torch.stack(got, 1)                      # [B, steps, Hq, d]
    pos = torch.arange(steps, device="cuda")
    for b in range(B):
        rq = fa2.norm_rope(q[:, b], qw, pos, freq).transpose(0, 1)[None].contiguous()
        rk = fa2.norm_rope(k[:, b], kw, pos, freq)
        rep = lambda t: t.repeat_interleave(Hq // Hkv, 1).transpose(0, 1)[None].contiguous()  # noqa: E731
        ref, _ = fa2.forward(rq, rep(rk), rep(v[:, b]), causal=True)
        # both sides round P and the paged one O: (2 u) A + u |O|, A <= max |v|
        u = EPS[BF]
        bound = 2.5 * u * v.abs().max().item() + u * ref.abs()
        assert ((got[b].transpose(0, 1)[None].float() - ref).abs() <= bound).all()


def test_other_streams_and_given_buffers():
    s = torch.cuda.Stream()
    x, dy = normal((1, 4, 1000, 128), BF, 1), normal((1, 4, 1000, 128), BF, 2)
    w, pos, freq = normal((128,), BF, 3), torch.arange(1000, device="cuda"), fa2.rope_inv_freq(128, device="cuda")
    y = fa2.norm_rope(x, w, pos, freq)
    dx, dw = fa2.norm_rope_backward(dy, x, w, pos, freq)
    size = fa2.library().fa2_norm_rope_backward_workspace_bytes(128)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        got = [fa2.norm_rope(x, w, pos, freq, stream=handle),
               *fa2.norm_rope_backward(dy, x, w, pos, freq, stream=handle),
               *fa2.norm_rope_backward(dy, x, w, pos, freq, dx=torch.empty_like(dx), dweight=torch.empty_like(dw),
                                       workspace=ws, stream=handle)]
        s.synchronize()
        for a, b in zip(got, (y, dx, dw, dx, dw)):
            assert torch.equal(a, b)
    with pytest.raises(fa2.FA2Error):
        fa2.norm_rope_backward(dy, x, w, pos, freq, workspace=ws[:size // 2].clone())


def test_rows_beyond_32_bits():
    """More than 2^31 elements: the rows at both ends and around the border."""
    H, N, d = 64, 270000, 128                     # 2.2e9 elements
    x = torch.empty((1, H, N, d), dtype=BF, device="cuda")
    y, freq, w = torch.empty_like(x), fa2.rope_inv_freq(d, device="cuda"), normal((d,), BF, 3, 0.3, 1.0)
    x.view(torch.int16).zero_()
    border = (1 << 31) // (N * d)
    places = [(0, 0), (border, (1 << 31) // d - border * N), (H - 1, N - 1), (H - 1, 5)]
    for i, (h, n) in enumerate(places):
        x[0, h, n] = normal((d,), BF, 10 + i)
    pos = torch.arange(N, device="cuda")
    assert fa2.norm_rope(x, w, pos, freq, out=y) is y
    for h, n in places:
        ref, bound, size = forward_64(x[0, h, n:n + 1], w, pos[n:n + 1], freq, 1e-6, False, 1.0)
        close(y[0, h, n:n + 1], ref, rounded(bound, size, BF))
    dx, dw = fa2.norm_rope_backward(x, x, w, pos, freq, dx=y)
    total, slacks = 0.0, 0.0
    for h, n in places:
        ref, bound, dw_, dw_bound = backward_64(x[0, h, n:n + 1], x[0, h, n:n + 1], w, pos[n:n + 1], freq, 1e-6, False,
                                                1.0, chain=8)
        close(dx[0, h, n:n + 1], ref, rounded(bound, ref, BF))
        total, slacks = total + dw_, slacks + dw_bound
    close(dw, total, slacks)                      # (all other rows are zeros)


def test_outputs_that_overlap_are_refused():
    buffer = normal((2, 8, 65, 128), BF, 1)
    w, pos, freq = normal((128,), BF, 3), torch.arange(64, device="cuda"), fa2.rope_inv_freq(128, device="cuda")
    x, shifted = buffer[:, :, :64], buffer[:, :, 1:]
    with pytest.raises(fa2.FA2Error):              # in place, but a row further
        fa2.norm_rope(x, w, pos, freq, out=shifted)
    with pytest.raises(fa2.FA2Error):
        fa2.norm_rope_backward(x, x, w, pos, freq, dx=shifted)
    with pytest.raises(fa2.FA2Error):              # rows of the output on one another
        fa2.norm_rope(x, w, pos, freq, out=torch.zeros((2, 1, 64, 128), dtype=BF, device="cuda").expand(2, 8, 64, 128))
    with pytest.raises(ValueError):
        fa2.norm_rope(x, w[:64], pos, freq)
    with pytest.raises(ValueError):
        fa2.norm_rope(x, w.half(), pos, freq)

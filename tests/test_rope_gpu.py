"""Rotary positions, their gradient, and new tokens written into a paged cache."""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, Cache, offsets, release_memory, rotate, rotate_bound

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


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def close(y, ref, bound):
    worst = ((y.double() - ref).abs() / (bound + 1e-30)).max() if y.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.3f} of the bound"


CASES = [
    # dtype, B, H, N, d, rotary, interleaved, first position
    (BF, 1, 1, 1, 64, 64, False, 0),
    (BF, 2, 3, 5, 128, 128, False, 7),
    (HF, 1, 8, 100, 128, 64, True, 1000),
    (F32, 2, 2, 33, 64, 48, True, 0),
    (F32, 2, 2, 33, 64, 48, False, 131071),
    (BF, 1, 40, 17, 256, 256, True, 1 << 20),
    (BF, 3, 5, 300, 128, 96, False, (1 << 31) - 400),
    (HF, 1, 2, 9, 80, 20, False, 3),            # halves that fill no vector
    (BF, 2, 2, 9, 80, 20, True, 3),
    (BF, 1, 3, 21, 66, 34, False, 11),          # rows that start off 16 bytes
    (HF, 1, 3, 21, 66, 34, True, 11),
    (F32, 1, 2, 10, 6, 2, False, 5),
    (BF, 1, 2, 10, 1024, 1024, False, 5),
    (BF, 1, 9, 4000, 64, 64, False, 100000),
    (BF, 1, 2, 50, 128, 128, False, -20),       # positions below zero
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}-{c[1]}x{c[2]}x{c[3]}x{c[4]}-r{c[5]}{'i' if c[6] else 'h'}")
@pytest.mark.parametrize("backward", [False, True])
def test_matches_the_64_bit_form(case, backward):
    dtype, B, H, N, d, r, interleaved, start = case
    x = normal((B, H, N, d), dtype, seed=N)
    freq = fa2.rope_inv_freq(r, device="cuda")
    pos = torch.arange(start, start + N, dtype=torch.int64 if start % 2 else torch.int32, device="cuda")
    call = fa2.rope_backward if backward else fa2.rope
    y = call(x, pos, freq, interleaved=interleaved, mscale=1.25)
    close(y, rotate(x, pos, freq, interleaved, 1.25, -1.0 if backward else 1.0),
          rotate_bound(x, freq, interleaved, dtype, 1.25))
    assert torch.equal(y[..., r:], x[..., r:])
    # in place
    z = x.clone()
    assert call(z, pos, freq, interleaved=interleaved, mscale=1.25, out=z) is z
    assert torch.equal(z, y)


def test_packed_tokens_strides_and_batched_positions():
    T, H, d = 77, 6, 128
    freq = fa2.rope_inv_freq(64, device="cuda")
    wide = normal((T, 3, H, d + 8), BF, seed=1)
    x = wide[:, 1, :, :d]
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(2)).to(torch.int32).cuda()
    ref = rotate(x.transpose(0, 1), pos, freq, False).transpose(0, 1)
    bound = rotate_bound(x, freq, False, BF)
    close(fa2.rope(x, pos, freq), ref, bound)
    out = torch.empty((H, T, d), dtype=BF, device="cuda").transpose(0, 1)
    close(fa2.rope(x, pos, freq, out=out), ref, bound)
    # positions of their own for each batch; a batch read twice
    x = normal((1, H, 30, d), BF, seed=3).expand(2, H, 30, d)
    pos = torch.stack([torch.arange(30), torch.arange(30) * 1000]).cuda()
    y = fa2.rope(x, pos, freq, interleaved=True)
    for b in range(2):
        close(y[b], rotate(x[b], pos[b], freq, True), rotate_bound(x[b], freq, True, BF))


def test_far_positions_keep_their_angle():
    """2^31 - 1 positions from zero the angle is still that of the 64-bit frequency (fp32 would be off by turns)."""
    freq = torch.tensor([1.0, 0.7, 1e-3, 1e-9], dtype=torch.float64, device="cuda")
    pos = torch.tensor([(1 << 31) - 1, 1999999999, 12345678, 3], device="cuda")
    x = torch.zeros((1, 1, 4, 8), dtype=F32, device="cuda")
    x[..., :4] = 1.0
    y = fa2.rope(x, pos, freq)[0, 0]
    # exact angle: 64-bit products of at most 2^31 * 2^-53 turns error, in Python's integers
    for i, t in enumerate(pos.tolist()):
        for j, f in enumerate(freq.tolist()):
            a = math.fmod(t * f, 2 * math.pi)
            assert abs(y[i, j].item() - math.cos(a)) < 1e-6 and abs(y[i, 4 + j].item() - math.sin(a)) < 1e-6


def test_gradient_against_differences():
    """d/dx of sum(w * rope(x)) by central differences; the map is linear, so in
    fp32 they carry rounding alone: 2 * 2^-22 * |values| / step."""
    x = normal((1, 2, 3, 16), F32, seed=4)
    w = normal((1, 2, 3, 16), F32, seed=5)
    freq = fa2.rope_inv_freq(8, device="cuda")
    pos = torch.tensor([5, 90, 4096], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        g = fa2.rope_backward(w, pos, freq, interleaved=interleaved, mscale=1.5)
        f = lambda t: (w.double() * fa2.rope(t, pos, freq, interleaved=interleaved, mscale=1.5).double()).sum()  # noqa: E731
        for e in range(0, x.numel(), 7):
            d = torch.zeros_like(x).view(-1)
            d[e] = 0.5
            d = d.view_as(x)
            diff = (f(x + d) - f(x - d)).item()
            assert abs(diff - g.view(-1)[e].item()) < 2e-5


def test_frequencies_of_long_contexts():
    plain = fa2.rope_inv_freq(64)
    assert plain.dtype == torch.float64 and plain[0] == 1.0 and abs(plain[16].item() - 1e-2) < 1e-15
    assert torch.equal(fa2.rope_inv_freq(64, scaling="linear", factor=4.0), plain / 4.0)
    base = fa2.rope_inv_freq(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and abs(base[-1] * 4.0 / plain[-1] - 1) < 1e-12
    ramp = fa2.rope_inv_freq(64, scaling="ramp", factor=4.0)
    assert torch.equal(ramp[:5], plain[:5]) and torch.equal(ramp[-5:], plain[-5:] / 4.0)
    assert ((ramp <= plain) & (ramp >= plain / 4.0)).all()


APPEND = [
    # dtype, d, Hq, Hkv, page, q lengths, lengths, rotary, interleaved
    (BF, 128, 8, 2, 16, [1, 1, 1], [1, 16, 17], 128, False),
    (HF, 64, 4, 4, 32, [5, 0, 40, 1], [5, 3, 100, 33], 32, True),
    (BF, 256, 6, 2, 64, [130, 7], [400, 7], 64, False),
    (BF, 128, 0, 3, 128, [9, 300], [9, 1000], 0, False),
    (HF, 128, 16, 1, 1024, [20, 3], [1500, 2000], 20, False),     # halves that fill no vector
    (BF, 64, 3, 3, 16, [10, 20], [4, 20], 64, True),              # more new tokens than the length
    (BF, 128, 32, 8, 16, [1] * 70, [(31 * i) % 500 + 1 for i in range(70)], 128, False),
]


@pytest.mark.parametrize("layout", ["phsd", "pshd", "layers"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{str(c[0])[6:]}-d{c[1]}-h{c[2]}.{c[3]}-s{c[4]}-r{c[7]}")
def test_append_writes_the_new_tokens_alone(case, layout):
    dtype, d, Hq, Hkv, S, q_lens, kv, r, interleaved = case
    cache = Cache(kv, Hkv, S, d, dtype, seed=5, layout=layout)
    T = sum(q_lens)
    k, v = normal((T + 3, Hkv, d), dtype, 6), normal((T + 3, Hkv, d), dtype, 7)
    q = normal((T + 3, Hq, d), dtype, 8) if Hq else None
    freq = fa2.rope_inv_freq(r, device="cuda") if r else None
    before_k, before_v = cache.k.clone(), cache.v.clone()
    q_out = None if q is None else torch.full_like(q, 7.0)
    got = fa2.append_paged(k, v, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens), q=q, q_out=q_out,
                           inv_freq=freq, interleaved=interleaved, mscale=1.25)
    assert got is q_out
    freq = torch.zeros(0, dtype=torch.float64, device="cuda") if freq is None else freq
    at = 0
    for b, (n, length) in enumerate(zip(q_lens, kv)):
        pos = torch.arange(length - n, length, device="cuda")
        rows = slice(at, at + n)
        at += n
        if q is not None:
            ref = rotate(q[rows].transpose(0, 1), pos, freq, interleaved, 1.25).transpose(0, 1)
            close(q_out[rows], ref, rotate_bound(q[rows], freq, interleaved, dtype, 1.25))
        there = pos >= 0
        pos, new_k, new_v = pos[there], k[rows][there], v[rows][there]
        page, slot = cache.table[b].long()[pos // S], pos % S
        ref = rotate(new_k.transpose(0, 1), pos, freq, interleaved, 1.25).transpose(0, 1)
        close(cache.k[page, :, slot], ref, rotate_bound(new_k, freq, interleaved, dtype, 1.25))
        assert torch.equal(cache.v[page, :, slot], new_v)
        before_k[page, :, slot] = cache.k[page, :, slot]
        before_v[page, :, slot] = new_v
    same = lambda a, b: torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))  # noqa: E731
    assert same(cache.k, before_k) and same(cache.v, before_v)
    assert q_out is None or (q_out[T:] == 7.0).all()


def test_append_outside_the_cache_is_reported_and_writes_nothing():
    cache = Cache([40, 20], 2, 16, 64, BF, seed=9)
    k, v = normal((2, 2, 64), BF, 1), normal((2, 2, 64), BF, 2)
    before = cache.k.clone()

    def status():
        torch.cuda.synchronize()
        return fa2.fa2_device_status(None, reset=True)

    for table, lens in ((torch.full_like(cache.table, -1), cache.lens),
                        (torch.full_like(cache.table, cache.k.shape[0]), cache.lens),
                        (cache.table, cache.lens + 16 * cache.table.shape[1])):
        fa2.append_paged(k, v, cache.k, cache.v, table, lens)
        assert status() == fa2.FA2_ERR_PAGE
        assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16))


def test_append_then_attend_as_a_step_does():
    """Prompt, then single tokens, through the cache: as attention over all keys at once."""
    d, Hq, Hkv, S, n, steps = 128, 8, 2, 16, 45, 7
    total = n + steps
    g = dict(dtype=BF)
    q, k, v = normal((total, Hq, d), g["dtype"], 1), normal((total, Hkv, d), BF, 2), normal((total, Hkv, d), BF, 3)
    freq = fa2.rope_inv_freq(d, device="cuda")
    pages = -(-total // S)
    kp, vp = (torch.full((pages, Hkv, S, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    out = []
    for first, last in [(0, n)] + [(i, i + 1) for i in range(n, total)]:
        add = torch.tensor([last - first], dtype=torch.int32, device="cuda")
        missing = fa2.pages_reserve(table, lens, refs, add, S)
        assert missing.item() == 0
        cu = None if last - first == 1 else offsets([last - first])
        rq = fa2.append_paged(k[first:last], v[first:last], kp, vp, table, lens, cu_q=cu, q=q[first:last],
                              inv_freq=freq)
        out.append(fa2.forward_paged(rq, kp, vp, table, lens, cu_q=cu)[0])
    got = torch.cat(out)
    pos = torch.arange(total, device="cuda", dtype=torch.int32)
    heads = lambda t: fa2.rope(t, pos, freq).transpose(0, 1)[None].contiguous()  # noqa: E731
    rep = lambda t: t.repeat_interleave(Hq // Hkv, 1)  # noqa: E731
    ref, _ = fa2.forward(heads(q), heads(rep(k)), rep(v).transpose(0, 1)[None].contiguous(), causal=True)
    # both sides round P and the paged one O: (2 u) A + u |O|, A <= max |v|
    u = EPS[BF]
    bound = 2.5 * u * v.abs().max().item() + u * ref.abs()
    assert ((got.transpose(0, 1)[None].float() - ref).abs() <= bound).all()


def test_other_streams():
    s = torch.cuda.Stream()
    x = normal((1, 4, 1000, 128), BF, 1)
    pos = torch.arange(1000, device="cuda", dtype=torch.int32)
    freq = fa2.rope_inv_freq(128, device="cuda")
    ref = fa2.rope(x, pos, freq)
    torch.cuda.synchronize()
    for handle in (s, s.cuda_stream):
        y = fa2.rope(x, pos, freq, stream=handle)
        s.synchronize()
        assert torch.equal(y, ref)

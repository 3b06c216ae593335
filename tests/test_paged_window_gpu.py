"""Attention over a paged cache with windows, and with prefixes that sequences share, against 64-bit forms."""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, Cache, offsets, release_memory
from window_reference import paged

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


def status():
    torch.cuda.synchronize()
    return fa2.fa2_device_status(None, reset=True)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def compare(got, ref, T):
    (o, lse), (ref, ref_lse, bO, bL) = got, ref
    none = ref_lse == -math.inf
    worst = ((o[:T].double() - ref).abs() / bO).max().item() if T else 0.0
    assert worst <= 1.0, f"O off by {worst:.3f} of the bound"
    assert torch.equal(lse[:T] == -math.inf, none) and (o[:T][none] == 0).all()
    off = ((lse[:T].double() - ref_lse).abs() / bL)[~none]
    assert not off.numel() or off.max() <= 1.0, f"LSE off by {off.max():.3f} of the bound"


def sees(n, length, window, sinks):
    i, j = torch.arange(length - n, length, device="cuda")[:, None], torch.arange(length, device="cuda")[None]
    return (j <= i) & ((i - j < window) | (j < sinks))


def forget(cache, q_lens, window, sinks):
    """Pages that no new token sees: their table entries outside the pool, or a page of NaN."""
    spare = cache.k.shape[0] - 1
    used = set(cache.table[cache.table < cache.k.shape[0]].tolist())
    nan_page = next(p for p in range(spare, -1, -1) if p not in used)
    gone = 0
    for b, (n, length) in enumerate(zip(q_lens, cache.kv)):
        lo = length - n - window + 1
        for page in range(-(-length // cache.S)):
            if (page + 1) * cache.S <= lo and page * cache.S >= sinks and n > 0:
                cache.table[b, page] = nan_page if page % 2 else (1 << 30) - page
                gone += 1
    return gone


WINDOW = [
    # dtype, d, Hq, Hkv, page, q lengths, lengths, window, sinks
    (BF, 128, 8, 2, 16, None, [1, 16, 17, 500, 3000, 0], 100, 4),        # single tokens
    (HF, 64, 4, 4, 64, None, [1000, 2000, 129, 128, 127], 1, 0),
    (BF, 256, 6, 2, 256, None, [5000, 300, 1200], 1000, 300),
    (BF, 128, 32, 1, 1024, None, [10000, 3, 2048], 130, 20),
    (HF, 128, 40, 1, 32, None, [3000] * 5, 400, 1),                      # groups of 40 heads
    (BF, 64, 8, 2, 16, [5, 0, 40, 1], [5, 3, 1000, 33], 64, 2),
    (BF, 128, 8, 2, 32, [300, 7, 129], [3000, 7, 700], 128, 4),
    (HF, 128, 4, 4, 128, [513, 100], [2000, 100], 300, 140),
    (BF, 256, 4, 1, 16, [100, 30], [1500, 2000], 200, 5),
    (BF, 64, 5, 1, 16, [10, 20], [4, 20], 3, 1),                         # more new tokens than the length
    (HF, 64, 8, 8, 512, [1000], [5000], 2000, 0),
    (BF, 128, 20, 4, 16, [1000, 1], [1000, 5000], 100000, 3),            # the window holds everything
    (BF, 128, 2, 1, 64, [700, 3, 64], [900, 2000, 1000], 5, 100000),     # so do the sinks
    (BF, 128, 64, 8, 16, [4] * 40, [(53 * i) % 3000 + 4 for i in range(40)], 500, 4),
]


@pytest.mark.parametrize("layout", ["phsd", "pshd"])
@pytest.mark.parametrize("case", WINDOW, ids=lambda c: f"{str(c[0])[6:]}-d{c[1]}-h{c[2]}.{c[3]}-s{c[4]}-w{c[7]}-k{c[8]}")
def test_window(case, layout):
    dtype, d, Hq, Hkv, S, q_lens, kv, window, sinks = case
    cu = None if q_lens is None else offsets(q_lens)
    q_lens = [1] * len(kv) if q_lens is None else q_lens
    cache = Cache(kv, Hkv, S, d, dtype, seed=3, layout=layout)
    forget(cache, q_lens, window, sinks)
    T = sum(q_lens)
    q = normal((T + (3 if cu is not None else 0), Hq, d), dtype, 1)
    masks = [sees(n, length, window, sinks) for n, length in zip(q_lens, kv)]
    scale = 1.0 / math.sqrt(d)
    for kind in (dtype, F32):
        out = torch.full(q.shape, 7.0, dtype=kind, device="cuda")
        got = fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens, window, sinks, cu_q=cu, out=out,
                                       out_dtype=kind)
        compare(got, paged(q, cache.keys, cache.values, q_lens, masks, scale, EPS[kind]), T)
        assert (out[T:] == 7.0).all()
    again = fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens, window, sinks, cu_q=cu)
    assert torch.equal(again[0][:T], fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens, window,
                                                              sinks, cu_q=cu)[0][:T])
    assert status() == fa2.FA2_OK


def test_many_items():
    """Blocks enough for whole items from a counter: 8 sequences, 16 heads apart, 2 sub-tiles a CTA."""
    for d, n in ((128, 1400), (256, 700)):
        q_lens, kv = [n] * 8, [n + 300 * i for i in range(8)]
        cache = Cache(kv, 16, 32, d, BF, seed=3)
        assert forget(cache, q_lens, 200, 4) > 0
        q = normal((sum(q_lens), 16, d), BF, 1)
        got = fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens, 200, 4, cu_q=offsets(q_lens))
        masks = [sees(n, length, 200, 4) for length in kv]
        compare(got, paged(q, cache.keys, cache.values, q_lens, masks, 1.0 / math.sqrt(d), EPS[BF]), sum(q_lens))
    assert status() == fa2.FA2_OK


@pytest.mark.parametrize("d, Hkv", [(64, 8), (128, 8), (256, 4)])
def test_few_waves_of_short_windows(d, Hkv):
    """Between one and two waves of ragged blocks, sequences without new tokens and short ones among them."""
    q_lens = [700, 0, 1, 1500, 256, 257, 900, 33, 2100, 0, 640, 5]
    kv = [n + 97 * i for i, n in enumerate(q_lens)]
    cache = Cache(kv, Hkv, 16, d, BF, seed=7)
    assert forget(cache, q_lens, 100, 4) > 0
    q = normal((sum(q_lens) + 2, Hkv, d), BF, 1)
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    got = fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens, 100, 4, cu_q=offsets(q_lens), out=out,
                                   out_dtype=BF)
    masks = [sees(n, length, 100, 4) for n, length in zip(q_lens, kv)]
    compare(got, paged(q, cache.keys, cache.values, q_lens, masks, 1.0 / math.sqrt(d), EPS[BF]), sum(q_lens))
    assert (out[sum(q_lens):] == 7.0).all() and status() == fa2.FA2_OK


def test_a_window_of_everything_is_plain_attention():
    q_lens, kv = [70, 1, 300], [500, 900, 300]
    cache = Cache(kv, 2, 16, 128, BF, seed=4)
    q, cu = normal((sum(q_lens), 8, 128), BF, 1), offsets(q_lens)
    plain = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    for window, sinks in ((900, 0), (1 << 40, 3), (1, 1 << 40)):
        got = fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens, window, sinks, cu_q=cu)
        assert (got[0].float() - plain[0].float()).abs().max() <= 2.0 ** -7 * plain[0].abs().max().item()
        assert (got[1] - plain[1]).abs().max() <= 1e-4


def test_pages_in_a_window_are_still_checked():
    cache = Cache([400], 2, 16, 64, BF, seed=9)
    q = normal((1, 4, 64), BF, 1)
    for page, bad in ((24, True), (23, True), (0, True), (5, False)):
        table = cache.table.clone()
        table[0, page] = -1
        fa2.forward_paged_window(q, cache.k, cache.v, table, cache.lens, 20, 3)
        assert status() == (fa2.FA2_ERR_PAGE if bad else fa2.FA2_OK), page
    fa2.forward_paged_window(q, cache.k, cache.v, cache.table, cache.lens + 10000, 20, 3)
    assert status() == fa2.FA2_ERR_PAGE


def test_window_slides_as_a_server_decodes():
    """Append and attention step by step, pages freed as they leave the window: as windowed attention over all at once."""
    d, Hq, Hkv, S, total, window, sinks = 64, 8, 2, 16, 150, 40, 3
    q, k, v = normal((total, Hq, d), BF, 1), normal((total, Hkv, d), BF, 2), normal((total, Hkv, d), BF, 3)
    pool = torch.full((2, 12, Hkv, S, d), float("nan"), dtype=BF, device="cuda")
    table = torch.full((1, 10), -1, dtype=torch.int32, device="cuda")
    out = []
    for t in range(total):
        page, lens = t // S, ints([t + 1])
        table[0, page] = page if page < 5 else 1 + (page - 1) % 4   # page 0 holds the sinks; four others in turn
        gone = page - 4
        if gone >= 1:
            table[0, gone] = -1
        assert (gone + 1) * S <= max(0, t - window + 1)   # (nobody sees it any more)
        fa2.append_paged(k[t:t + 1], v[t:t + 1], pool[0], pool[1], table, lens)
        out.append(fa2.forward_paged_window(q[t:t + 1], pool[0], pool[1], table, lens, window, sinks)[0])
    heads = lambda t: t.transpose(0, 1)[None].contiguous()  # noqa: E731
    ref, _ = fa2.forward_window(heads(q), heads(k), heads(v), window, sinks)
    got = heads(torch.cat(out)).float()
    # both sides round P and the paged one O: (2 u) A + u |O|, A <= max |v|
    assert ((got - ref).abs() <= 2.5 * EPS[BF] * v.abs().max().item() + EPS[BF] * ref.abs()).all()
    assert status() == fa2.FA2_OK


# ---------------------------------------------------------------- shared prefixes

def share(cache, cu_groups, prefix_lens):
    """The groups' whole shared pages become those of their first sequences; the others' own copies become NaN."""
    S = cache.S
    for g, n in enumerate(prefix_lens):
        first, last = cu_groups[g], cu_groups[g + 1]
        pages = n // S
        for b in range(first + 1, last):
            old = cache.table[b, :pages].long()
            cache.k[old], cache.v[old] = float("nan"), float("nan")
            cache.table[b, :pages] = cache.table[first, :pages]
            for x in (cache.keys, cache.values):
                x[b][:pages * S] = x[first][:pages * S]


PREFIX = [
    # dtype, d, Hq, Hkv, page, q lengths, lengths, cu_groups, prefix_lens, causal
    (BF, 128, 8, 2, 16, None, [300, 310, 401], [0, 3], [288], True),
    (HF, 64, 4, 4, 64, None, [1000, 2000, 129, 128, 700], [0, 2, 2, 4], [960, 0, 127], True),   # an empty group, one outside
    (BF, 256, 6, 2, 32, None, [600, 513, 513], [1, 3], [512], True),              # one token of its own
    (BF, 128, 32, 1, 256, None, [5000, 4900, 4864, 10], [0, 3, 4], [4863, 3], True),   # a prefix that fills no page
    (HF, 128, 32, 8, 16, None, [2000 + i for i in range(40)], [0, 40], [1999], True),
    (BF, 64, 8, 2, 16, [5, 0, 40, 1], [205, 203, 1000, 233], [0, 4], [200], True),
    (BF, 128, 8, 2, 128, [300, 7, 129], [1000, 707, 829], [0, 2, 3], [700, 500], True),
    (HF, 128, 4, 4, 16, [64, 64, 64], [500, 600, 700], [0, 3], [400], False),     # every token sees everything
    (BF, 256, 4, 1, 16, [100, 30], [1500, 2000], [0, 2], [1400], True),
    (BF, 64, 40, 1, 1024, [3, 5, 2], [2100, 3000, 2200], [0, 3], [2050], True),
    (BF, 128, 8, 8, 16, [1] * 70, [(31 * i) % 500 + 600 for i in range(70)], [0, 20, 21, 60], [512, 600, 599], True),
    (HF, 64, 16, 4, 64, [2, 17, 9, 33] * 6, [9000 + 37 * i for i in range(24)], [0, 24], [8900], True),
    (BF, 128, 4, 2, 16, [0, 0, 3], [40, 40, 50], [0, 2, 3], [32, 16], True),      # a group without new tokens
]


@pytest.mark.parametrize("layout", ["phsd", "pshd"])
@pytest.mark.parametrize("case", PREFIX, ids=lambda c: f"{str(c[0])[6:]}-d{c[1]}-h{c[2]}.{c[3]}-s{c[4]}-b{len(c[6])}-p{c[8][0]}")
def test_prefix(case, layout):
    dtype, d, Hq, Hkv, S, q_lens, kv, cu_groups, prefix_lens, causal = case
    cu = None if q_lens is None else offsets(q_lens)
    q_lens = [1] * len(kv) if q_lens is None else q_lens
    cache = Cache(kv, Hkv, S, d, dtype, seed=3, layout=layout)
    share(cache, cu_groups, prefix_lens)
    T = sum(q_lens)
    q = normal((T + (3 if cu is not None else 0), Hq, d), dtype, 1)
    every = 1 << 30
    masks = [sees(n, length, every, 0) if causal else torch.ones(n, length, dtype=torch.bool, device="cuda")
             for n, length in zip(q_lens, kv)]
    how = dict(cu_q=cu, causal=causal)
    args = (q, cache.k, cache.v, cache.table, cache.lens, ints(cu_groups), ints(prefix_lens))
    for kind in (dtype, F32):
        out, lse = (torch.full(s, 7.0, dtype=t, device="cuda") for s, t in ((q.shape, kind), (q.shape[:2], F32)))
        got = fa2.forward_paged_prefix(*args, **how, out=out, lse=lse, out_dtype=kind)
        compare(got, paged(q, cache.keys, cache.values, q_lens, masks, 1.0 / math.sqrt(d), EPS[kind], parts=2), T)
        assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()
    one, two = fa2.forward_paged_prefix(*args, **how), fa2.forward_paged_prefix(*args, **how)
    assert torch.equal(one[0][:T], two[0][:T]) and torch.equal(one[1][:T], two[1][:T])
    assert status() == fa2.FA2_OK


def test_no_groups_is_plain_attention():
    cache = Cache([300, 20], 2, 16, 64, BF, seed=4)
    q = normal((2, 4, 64), BF, 1)
    plain = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens)
    got = fa2.forward_paged_prefix(q, cache.k, cache.v, cache.table, cache.lens, ints([0]), ints([]))
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    # groups of one share nothing: the same sums
    got = fa2.forward_paged_prefix(q, cache.k, cache.v, cache.table, cache.lens, ints([0, 1, 2]), ints([256, 16]))
    assert torch.equal(got[1], plain[1]) and torch.equal(got[0], plain[0])


def test_groups_out_of_order_are_reported():
    cache = Cache([300, 320, 310], 2, 16, 64, BF, seed=4)
    share(cache, [0, 3], [288])
    q = normal((3, 4, 64), BF, 1)
    call = lambda cu, lens: fa2.forward_paged_prefix(q, cache.k, cache.v, cache.table, cache.lens, ints(cu), ints(lens))  # noqa: E731
    call([0, 3], [288])
    assert status() == fa2.FA2_OK
    for cu, lens in (([0, 4], [288]), ([-1, 3], [288]), ([0, 3], [-5]), ([0, 3], [1 << 20]), ([2, 1], [16]),
                     ([0, 3], [304])):            # (a prefix beyond the shortest sequence's new token)
        call(cu, lens)
        assert status() == fa2.FA2_ERR_PAGE, (cu, lens)


def test_more_new_tokens_than_positions_beside_groups():
    """Sequences that share nothing (outside all groups, alone in one, or in one without a prefix) are plain attention's."""
    q_lens, kv = [5, 3, 3, 9, 40, 2], [4, 100, 110, 2, 30, 1]
    for cu_groups, prefix_lens in (([1, 3, 4], [96, 0]), ([1, 3, 3, 6], [96, 0, 0])):
        cache = Cache(kv, 2, 16, 64, BF, seed=5)
        share(cache, cu_groups, prefix_lens)
        q = normal((sum(q_lens), 8, 64), BF, 1)
        got = fa2.forward_paged_prefix(q, cache.k, cache.v, cache.table, cache.lens, ints(cu_groups), ints(prefix_lens),
                                       cu_q=offsets(q_lens), out_dtype=F32)
        masks = [sees(n, length, 1 << 30, 0) for n, length in zip(q_lens, kv)]
        compare(got, paged(q, cache.keys, cache.values, q_lens, masks, 0.125, EPS[F32], parts=2), sum(q_lens))
        assert status() == fa2.FA2_OK


def test_samples_of_one_prompt():
    """A prompt, forked into samples (pages_fork), then steps of append and attention with the prompt shared, captured
    and replayed: as attention without sharing."""
    d, Hq, Hkv, S, n, samples, steps = 128, 8, 2, 16, 200, 4, 20
    pool = torch.zeros((2, 64, Hkv, S, d), dtype=BF, device="cuda")
    table = torch.full((samples, 16), -1, dtype=torch.int32, device="cuda")
    lens, refs = ints([0] * samples), ints([0] * 64)
    prompt = [normal((n, h, d), BF, i) for i, h in enumerate((Hq, Hkv, Hkv))]
    assert fa2.pages_reserve(table, lens, refs, ints([n] + [0] * (samples - 1)), S).item() == 0
    fa2.append_paged(prompt[1], prompt[2], pool[0], pool[1], table[:1], lens[:1], cu_q=ints([0, n]))
    assert fa2.pages_fork(table, lens, refs, ints([0] * (samples - 1)), ints(list(range(1, samples))), pool).item() == 0
    cu, shared, one = ints([0, samples]), ints([n]), ints([1] * samples)
    now = [normal((samples, h, d), BF, 9) for h in (Hq, Hkv, Hkv)]

    def step():
        fa2.pages_reserve(table, lens, refs, one, S)
        fa2.append_paged(now[1], now[2], pool[0], pool[1], table, lens)
        return (*fa2.forward_paged_prefix(now[0], pool[0], pool[1], table, lens, cu, shared),
                *fa2.forward_paged(now[0], pool[0], pool[1], table, lens))

    saved = [t.clone() for t in (table, lens, refs)]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        for t, x in zip((table, lens, refs), saved):
            t.copy_(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step()
    for i in range(steps):
        for t, h in zip(now, (Hq, Hkv, Hkv)):
            t.copy_(normal((samples, h, d), BF, 100 + i))
        graph.replay()
        o, lse, ref, ref_lse = out
        # both sides round P and O
        assert ((o.float() - ref.float()).abs() <= 2.5 * EPS[BF] * 5 + 2 * EPS[BF] * ref.float().abs()).all()
        assert (lse - ref_lse).abs().max() <= 1e-4
    assert lens.tolist() == [n + steps] * samples and status() == fa2.FA2_OK


def test_streams_and_given_buffers():
    cache = Cache([700, 710, 720], 2, 16, 128, BF, seed=4)
    share(cache, [0, 3], [688])
    q, cu, lens = normal((3, 8, 128), BF, 1), ints([0, 3]), ints([688])
    args = (q, cache.k, cache.v, cache.table, cache.lens)
    ref, win = fa2.forward_paged_prefix(*args, cu, lens), fa2.forward_paged_window(*args, 100, 4)
    f = fa2.library()
    ws = torch.empty(f.fa2_forward_paged_prefix_workspace_bytes(3, 1, 3, 8, 2, 128, 0), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        got = fa2.forward_paged_prefix(*args, cu, lens, workspace=ws, stream=handle)
        got += fa2.forward_paged_window(*args, 100, 4, stream=handle)
        s.synchronize()
        for a, b in zip(got, (*ref, *win)):
            assert torch.equal(a, b)
    with pytest.raises(fa2.FA2Error):
        fa2.forward_paged_prefix(*args, cu, lens, workspace=ws[:1024].clone())


def test_a_cache_beyond_32_bits():
    """Pages behind 2^31 elements, windows and shared prefixes."""
    d, Hkv, S = 64, 4, 16
    P = (1 << 31) // (Hkv * S * d) + 64
    pages = [torch.empty((P, Hkv, S, d), dtype=BF, device="cuda") for _ in range(2)]
    kv = [300, 320, 310]
    small = Cache(kv, Hkv, S, d, BF, seed=5)
    share(small, [0, 3], [288])
    n = small.k.shape[0]
    for big, own in zip(pages, (small.k, small.v)):
        big[P - n:] = own
    table = torch.where(small.table < n, small.table + (P - n), small.table)
    q = normal((3, 8, d), BF, 1)
    for call in (lambda k, v, t: fa2.forward_paged_window(q, k, v, t, small.lens, 100, 4),
                 lambda k, v, t: fa2.forward_paged_prefix(q, k, v, t, small.lens, ints([0, 3]), ints([288]))):
        a, b = call(*pages, table), call(small.k, small.v, small.table)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert status() == fa2.FA2_OK

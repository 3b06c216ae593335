"""Attention over a paged cache against its 64-bit form."""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, Cache, attention, offsets, release_memory

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    libbuild.build()
    fa2.fa2_device_status(None, reset=True)
    yield
    assert fa2.fa2_device_status(None, reset=True) == fa2.FA2_OK
    release_memory()


def queries(q_lens, Hq, d, dtype, seed, std=1.0, tail=0):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn(sum(q_lens) + tail, Hq, d, generator=g) * std).to(dtype).cuda()


def check(o, lse, q, cache, q_lens, causal, scale, out_dtype=None):
    dtype = q.dtype
    n = sum(q_lens)
    O, L, bO, bL = attention(q[:n], cache.keys, cache.values, q_lens, causal, scale, dtype,
                             EPS[out_dtype or o.dtype])
    assert torch.equal(lse[:n].double() == -math.inf, L == -math.inf)
    live = L != -math.inf
    assert not torch.isnan(o[:n]).any() and not torch.isnan(lse[:n]).any()
    assert (o[:n][~live] == 0).all()
    worst = ((o[:n].double() - O).abs() / bO)[live]
    worst_l = ((lse[:n].double() - L).abs() / bL)[live]
    assert worst.numel() == 0 or worst.max() <= 1.0, f"O off by {worst.max():.3f} of its bound"
    assert worst_l.numel() == 0 or worst_l.max() <= 1.0, f"LSE off by {worst_l.max():.3f} of its bound"


CASES = [
    # dtype, d, Hq, Hkv, page, q lengths, lengths, causal
    (BF, 128, 8, 2, 16, [1], [1], True),
    (BF, 128, 8, 2, 16, [1, 1, 1], [1, 16, 17], True),
    (BF, 128, 8, 8, 16, [1, 1], [129, 1000], True),
    (HF, 64, 8, 1, 32, [1, 1, 1, 1], [0, 127, 128, 129], True),
    (BF, 256, 4, 2, 64, [1, 1], [300, 64], True),
    (BF, 128, 32, 8, 16, [1] * 40, [(37 * i) % 700 + 1 for i in range(40)], True),
    (HF, 64, 16, 16, 128, [5, 0, 17, 1], [5, 0, 1000, 129], True),
    (BF, 128, 12, 4, 32, [33, 70, 2], [40, 700, 2], True),       # three heads a group
    (BF, 128, 10, 2, 64, [130, 1, 64], [400, 513, 64], True),    # five
    (HF, 128, 14, 2, 16, [50, 19], [50, 333], True),             # seven
    (BF, 64, 17, 1, 16, [9, 31], [100, 31], True),               # seventeen: seven tokens a sub-tile
    (BF, 128, 128, 1, 256, [3, 2], [700, 2], True),              # one token a sub-tile
    (BF, 128, 4, 4, 1024, [300, 129], [1500, 129], True),        # two sub-tiles a block
    (BF, 64, 4, 4, 512, [257, 600, 1], [2000, 600, 900], True),
    (HF, 256, 6, 2, 128, [200, 77], [600, 77], True),
    (BF, 128, 8, 2, 16, [90, 20], [60, 5], True),                # more new tokens than keys: empty rows
    (BF, 128, 4, 4, 32, [300, 280], [100, 0], True),             # whole blocks without a key
    (BF, 128, 8, 2, 16, [90, 20, 4], [60, 5, 0], False),
    (BF, 128, 4, 4, 64, [300, 513], [1000, 70], False),
    (HF, 256, 8, 2, 32, [40, 3], [513, 1], False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}-d{c[1]}-h{c[2]}.{c[3]}-s{c[4]}-{'c' if c[7] else 'n'}-{c[5][:3]}")
def test_matches_the_64_bit_form(case):
    dtype, d, Hq, Hkv, S, q_lens, kv, causal = case
    cache = Cache(kv, Hkv, S, d, dtype, seed=d + len(kv))
    q = queries(q_lens, Hq, d, dtype, seed=Hq)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens), causal=causal)
    check(o, lse, q, cache, q_lens, causal, 1 / math.sqrt(d))


@pytest.mark.parametrize("d,Hq,Hkv,S", [(64, 8, 2, 16), (128, 32, 4, 16), (128, 3, 3, 64), (256, 16, 1, 256)])
def test_single_tokens_without_offsets(d, Hq, Hkv, S):
    kv = [1, 15, 16, 128, 129, 0, 2500, 777]
    cache = Cache(kv, Hkv, S, d, BF, seed=1)
    q = queries([1] * 8, Hq, d, BF, seed=2)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens)
    check(o, lse, q, cache, [1] * 8, True, 1 / math.sqrt(d))
    # the same through offsets
    o2, lse2 = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets([1] * 8))
    check(o2, lse2, q, cache, [1] * 8, True, 1 / math.sqrt(d))


@pytest.mark.parametrize("d,dtype,q_lens,kv", [(128, BF, [1], [20000]), (64, HF, [1, 3], [30000, 9]),
                                               (128, BF, [300], [9000]), (256, BF, [2, 40], [12000, 700])])
def test_long_sequences_are_cut_into_ranges(d, dtype, q_lens, kv):
    """Few rows over many keys: the ranges' results are merged, to the same bits every time."""
    cache = Cache(kv, 2, 64, d, dtype, seed=3)
    q = queries(q_lens, 8, d, dtype, seed=4, std=3.0)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens))
    check(o, lse, q, cache, q_lens, True, 1 / math.sqrt(d))
    o2, lse2 = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_peaked_scores_move_the_offset():
    """Keys whose scores grow along the sequence, far past the softmax offset's step."""
    d, kv = 128, [1500]
    cache = Cache(kv, 1, 32, d, BF, seed=5)
    scale = torch.linspace(0.1, 8.0, kv[0], device="cuda").to(BF)
    k = cache.keys[0] * scale[:, None, None]
    pos = torch.arange(kv[0], device="cuda")
    page = cache.table[0].long()[pos // 32]
    cache.k[page, :, pos % 32] = k
    cache.keys[0] = k
    q = queries([64], 4, d, BF, seed=6, std=4.0)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets([64]))
    check(o, lse, q, cache, [64], True, 1 / math.sqrt(d))


@pytest.mark.parametrize("layout", ["pshd", "layers"])
@pytest.mark.parametrize("S", [16, 128])
def test_other_layouts_and_strided_queries(layout, S):
    q_lens, kv, d = [7, 1, 140], [300, 77, 200], 128
    cache = Cache(kv, 2, S, d, BF, seed=7, layout=layout)
    n = sum(q_lens)
    wide = torch.full((n, 3, 6, d + 8), float("nan"), dtype=BF, device="cuda")   # q inside a wider projection
    q = wide[:, 1, :, :d]
    q.copy_(queries(q_lens, 6, d, BF, seed=8))
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens), scale=0.05)
    check(o, lse, q, cache, q_lens, True, 0.05)


def test_outputs_in_32_bits_and_rows_of_nobody():
    q_lens, kv, d = [3, 130], [50, 300], 128
    cache = Cache(kv, 4, 32, d, BF, seed=9)
    q = queries(q_lens, 8, d, BF, seed=10, tail=6)
    out = torch.full((139, 8, d), 7.0, device="cuda")
    lse = torch.full((139, 8), 7.0, device="cuda")
    o, l2 = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens), out=out, lse=lse,
                              out_dtype=torch.float32)
    assert o is out and l2 is lse
    check(o, lse, q, cache, q_lens, True, 1 / math.sqrt(d), torch.float32)
    assert (out[133:] == 7.0).all() and (lse[133:] == 7.0).all()
    # no query at all: nothing happens
    o, lse = fa2.forward_paged(q[:0], cache.k, cache.v, cache.table, cache.lens, cu_q=offsets([0, 0]))
    assert o.shape == (0, 8, d)


def test_slots_past_32_bits():
    """A pool whose last pages lie more than 2^32 bytes and elements in."""
    d, S, Hkv = 128, 128, 8
    P = (1 << 32) // (S * Hkv * d) + 9
    k = torch.empty((P, Hkv, S, d), dtype=BF, device="cuda")
    v = torch.empty((P, Hkv, S, d), dtype=BF, device="cuda")
    kv = [500]
    small = Cache(kv, Hkv, S, d, BF, seed=11, spare=0)
    table = torch.tensor([[P - 1, 0, P - 2, P - 5]], dtype=torch.int32, device="cuda")
    for i in range(4):
        k[table[0, i]] = small.k[small.table[0, i]]
        v[table[0, i]] = small.v[small.table[0, i]]
    q = queries([3], 16, d, BF, seed=12)
    o, lse = fa2.forward_paged(q, k, v, table, small.lens, cu_q=offsets([3]))
    check(o, lse, q, small, [3], True, 1 / math.sqrt(d))


def test_captured_call_follows_lengths_and_tables():
    d, Hq, Hkv, S = 128, 8, 2, 16
    kv = [700, 40, 333]
    cache = Cache(kv, Hkv, S, d, BF, seed=13)
    q = queries([1] * 3, Hq, d, BF, seed=14)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens)
    lens = cache.lens.clone()
    out, l2 = torch.empty_like(o), torch.empty_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa2.forward_paged(q, cache.k, cache.v, cache.table, lens, out=out, lse=l2)
    graph.replay()
    assert torch.equal(out, o) and torch.equal(l2, lse)
    lens.copy_(torch.tensor([650, 0, 17], device="cuda"))
    graph.replay()
    cut = Cache(kv, Hkv, S, d, BF, seed=13)
    cut.keys = [k[:n] for k, n in zip(cut.keys, [650, 0, 17])]
    cut.values = [v[:n] for v, n in zip(cut.values, [650, 0, 17])]
    check(out, l2, q, cut, [1] * 3, True, 1 / math.sqrt(d))


def test_two_streams_at_once():
    d = 64
    caches = [Cache([9000, 300], 2, 32, d, BF, seed=s) for s in (15, 16)]
    qs = [queries([2, 40], 8, d, BF, seed=s) for s in (17, 18)]
    cu = offsets([2, 40])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    results = []
    for _ in range(3):
        for c, q, s in zip(caches, qs, streams):
            results.append((c, q, fa2.forward_paged(q, c.k, c.v, c.table, c.lens, cu_q=cu, stream=s)))
    torch.cuda.synchronize()
    for c, q, (o, lse) in results:
        check(o, lse, q, c, [2, 40], True, 1 / math.sqrt(d))


def test_two_captured_calls_on_two_streams():
    """Each capture has its own workspace: replays may overlap each other and an eager call."""
    d = 128
    cu = offsets([3, 50])
    calls = []
    for s in range(2):
        cache = Cache([7000, 900], 2, 32, d, BF, seed=30 + s)
        q = queries([3, 50], 8, d, BF, seed=40 + s)
        fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
        calls.append((cache, q, graph, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        for cache, q, graph, out, stream in calls:
            with torch.cuda.stream(stream):
                graph.replay()
        eager = fa2.forward_paged(calls[0][1], calls[0][0].k, calls[0][0].v, calls[0][0].table, calls[0][0].lens, cu_q=cu)
    torch.cuda.synchronize()
    for cache, q, graph, (o, lse), stream in calls:
        check(o, lse, q, cache, [3, 50], True, 1 / math.sqrt(d))
    assert torch.equal(eager[0], calls[0][3][0])


def test_given_outputs_and_workspace_are_checked_and_used():
    d = 64
    cache = Cache([5000, 30], 2, 16, d, BF, seed=23)
    q = queries([1, 1], 8, d, BF, seed=24)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens)     # the compiled binding
    need = fa2.library().fa2_forward_paged_workspace_bytes(2, 2, 8, 2, d, 0)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ws.fill_(255)                                                                  # NaN everywhere
    given = [torch.empty_like(o), torch.empty_like(lse)]
    fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, out=given[0], lse=given[1], workspace=ws)
    assert torch.equal(given[0], o) and torch.equal(given[1], lse)
    args = (q, cache.k, cache.v, cache.table, cache.lens)
    with pytest.raises(fa2.FA2Error) as e:
        fa2.forward_paged(*args, workspace=ws[:need - 256])
    assert e.value.status == fa2.FA2_ERR_MEMORY
    for bad in (dict(out=o.float()), dict(out=o[:1]), dict(lse=lse.half()), dict(out_dtype=HF), dict(cu_q=cache.lens),
                dict(workspace=ws[::2])):
        with pytest.raises(ValueError):
            fa2.forward_paged(*args, **bad)
    for bad in ((q[:, :7], *args[1:]), (q[:1], *args[1:]), (q.half(), *args[1:]), (q, cache.k, cache.v.half(), *args[3:]),
                (q, cache.k[..., :32], cache.v[..., :32], *args[3:]), (*args[:3], cache.table.long(), cache.lens),
                (*args[:3], cache.table[:1], cache.lens), (*args[:4], cache.lens.cpu())):
        with pytest.raises(ValueError):
            fa2.forward_paged(*bad)
    with pytest.raises(fa2.FA2Error) as e:
        fa2.forward_paged(*args, scale=0.0)
    assert e.value.status == fa2.FA2_ERR_SCALE
    odd = torch.empty((4, 2, 24, d), dtype=BF, device="cuda")                      # 24 slots a page
    with pytest.raises(fa2.FA2Error) as e:
        fa2.forward_paged(q, odd, odd, cache.table, cache.lens)
    assert e.value.status == fa2.FA2_ERR_SHAPE


def test_numbers_outside_the_cache_are_reported():
    d = 128
    cache = Cache([300, 40], 2, 16, d, BF, seed=19)
    q = queries([1, 1], 4, d, BF, seed=20)

    def status():
        torch.cuda.synchronize()
        return fa2.fa2_device_status(None, reset=True)

    assert status() == fa2.FA2_OK
    table = cache.table.clone()
    table[0, 3] = -1
    fa2.forward_paged(q, cache.k, cache.v, table, cache.lens)
    assert status() == fa2.FA2_ERR_PAGE
    table[0, 3] = cache.k.shape[0]
    fa2.forward_paged(q, cache.k, cache.v, table, cache.lens)
    assert status() == fa2.FA2_ERR_PAGE
    lens = cache.lens.clone()
    lens[0] = cache.table.shape[1] * 16 + 1
    fa2.forward_paged(q, cache.k, cache.v, cache.table.clamp(max=cache.k.shape[0] - 1), lens)
    assert status() == fa2.FA2_ERR_PAGE
    cu = torch.tensor([0, 1, 5], dtype=torch.int32, device="cuda")
    fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    assert status() == fa2.FA2_ERR_PAGE
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens)
    assert status() == fa2.FA2_OK
    check(o, lse, q, cache, [1, 1], True, 1 / math.sqrt(d))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 3, 40, 400])
def test_no_wait_runs_out(d, q_len):
    """Every wait in the kernels gives up after two seconds; none gets there."""
    cache = Cache([3000, 1500, 700], 2, 32, d, BF, seed=21)
    q_lens = [q_len] * 3
    q = queries(q_lens, 8, d, BF, seed=22)
    cu = offsets(q_lens)
    fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    first, last = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    first.record()
    fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    last.record()
    torch.cuda.synchronize()
    assert first.elapsed_time(last) < 500.0


def serve(steps, group, sync):
    """Dependent calls: room, append, attention, whose output makes the next step's tokens; forks between."""
    d, Hq, Hkv, S, B = 64, 8, 2, 16, 6
    g = torch.Generator().manual_seed(77)
    pool = torch.full((2, 256, Hkv, S, d), float("nan"), dtype=BF, device="cuda")
    table = torch.full((B, 40), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.int32, device="cuda")
    x = torch.randn(B * group, Hq, d, generator=g).to(BF).cuda()
    cu = offsets([group] * B) if group > 1 else None
    add = torch.full((B,), group, dtype=torch.int32, device="cuda")
    freq = fa2.rope_inv_freq(d, device="cuda")
    src, dst = (torch.tensor([i], dtype=torch.int32, device="cuda") for i in (0, 5))
    wait = torch.cuda.synchronize if sync else (lambda: None)
    wait()
    seen = []
    for step in range(steps):
        if step % 4 == 3:
            fa2.pages_free(table, lens, refs, dst)
            wait()
            fa2.pages_fork(table, lens, refs, src, dst, (pool[0], pool[1]))
            wait()
        missing = fa2.pages_reserve(table, lens, refs, add, S)
        wait()
        q = fa2.append_paged(x[:, :Hkv], x[:, Hkv:2 * Hkv], pool[0], pool[1], table, lens, cu, q=x, inv_freq=freq)
        wait()
        o, lse = fa2.forward_paged(q, pool[0], pool[1], table, lens, cu_q=cu)
        wait()
        x = fa2.rope(o.transpose(0, 1).unsqueeze(0), torch.arange(B * group, device="cuda"),
                     freq)[0].transpose(0, 1).contiguous() if step % 2 else o
        wait()
        seen += [missing, q, o, lse]
    torch.cuda.synchronize()
    return seen + [table, lens, refs]


@pytest.mark.parametrize("group", [1, 7])
def test_dependent_calls_without_waits_between(group):
    """Kernels start behind one another: the same bits as with the device idle between calls."""
    want = serve(24, group, True)
    for _ in range(3):
        for a, b in zip(serve(24, group, False), want):
            assert torch.equal(a, b)


def test_captured_chain_of_many_blocks():
    """Whole items from the counter in the workspace, replayed: the counter starts over every time."""
    d, Hq, Hkv = 128, 16, 16
    q_lens, kv = [2100, 8000], [2500, 8000]
    cache = Cache(kv, Hkv, 64, d, BF, seed=50)
    q = queries(q_lens, Hq, d, BF, seed=51)
    cu = offsets(q_lens)
    want = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
        second = fa2.forward_paged(first[0], cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    chained = fa2.forward_paged(want[0], cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first + second, want + chained):
        assert torch.equal(a, b)
    rows = [0, 1, 2099]
    O, L, bO, bL = attention(q[:2100], cache.keys[:1], cache.values[:1], [2100], True, 1 / math.sqrt(d), BF, EPS[BF])
    assert ((want[0][rows].double() - O[rows]).abs() <= bO[rows]).all()
    assert ((want[1][rows].double() - L[rows]).abs() <= bL[rows]).all()


def test_captured_behind_a_copy_and_another_stream():
    """The node before a call may be a copy or a clearing, and another stream's work may join."""
    d, Hq, Hkv = 128, 8, 2
    cache = Cache([700, 40, 333], Hkv, 16, d, BF, seed=60)
    q = queries([1] * 3, Hq, d, BF, seed=61)
    want = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens)
    freq = fa2.rope_inv_freq(d, device="cuda")
    pos = torch.arange(3, device="cuda")
    turned = fa2.rope(q, pos, freq)
    lens, q2, q3 = torch.zeros_like(cache.lens), torch.zeros_like(q), torch.zeros_like(q)
    scratch = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q2.copy_(q)
            r2 = fa2.rope(q2, pos, freq)
        lens.copy_(cache.lens)
        scratch.zero_()
        q3.copy_(q)
        got = fa2.forward_paged(q3, cache.k, cache.v, cache.table, lens)
        main.wait_stream(side)
        r3 = fa2.rope(r2, pos * 0, freq)            # behind both streams
        again = fa2.forward_paged(q2, cache.k, cache.v, cache.table, lens)
    for _ in range(3):
        lens.zero_()
        q2.zero_()
        q3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + again, want + want):
            assert torch.equal(a, b)
        assert torch.equal(r2, turned) and torch.equal(r3, turned)


@pytest.mark.parametrize("B", [33, 64, 1025, 2100])
@pytest.mark.parametrize("chunks", [False, True])
def test_many_short_sequences(B, chunks):
    """The schedule's strips of sequences: more than one each, and more than 32."""
    d, Hq, Hkv, S = 64, 4, 2, 16
    kv = [(53 * i) % 40 if i % 9 else 0 for i in range(B)]
    q_lens = [(i % 3) if chunks else 1 for i in range(B)]
    kv = [max(n, c) for n, c in zip(kv, q_lens)] if chunks else kv
    cache = Cache(kv, Hkv, S, d, BF, seed=70)
    q = queries(q_lens, Hq, d, BF, seed=71)
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens) if chunks else None)
    check(o, lse, q, cache, q_lens, True, 1 / math.sqrt(d))

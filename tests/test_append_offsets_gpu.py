"""Lengths and offsets outside the cache: an append reports them and writes nothing for their sequences."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import Cache, release_memory

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
D, HKV, S = 64, 2, 16


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    libbuild.build()
    fa2.fa2_device_status(None, reset=True)
    yield
    assert fa2.fa2_device_status(None, reset=True) == fa2.FA2_OK
    release_memory()


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def same(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# the sequences' lengths that the pages are made for; lengths and offsets of the call, tokens;
# (sequence, its first row, its first position, how many) of those that are in order
CASES = {
    "in order": ([40, 20], [40, 20], None, 2, [(0, 0, 39, 1), (1, 1, 19, 1)]),
    "end behind the tokens": ([40, 20], [40, 20], [0, 1, 5], 2, [(0, 0, 39, 1)]),
    "all of a sequence behind the tokens": ([40, 20, 33], [40, 20, 33], [0, 2, 7, 9], 2, [(0, 0, 38, 2)]),
    "begin below zero": ([40, 20], [40, 20], [-2, 1, 2], 2, [(1, 1, 19, 1)]),
    "all of a sequence below zero": ([40, 20], [40, 20], [-3, -1, 1], 1, []),
    "descending": ([60, 40, 50], [60, 40, 50], [0, 5, 3, 8], 8, [(0, 0, 55, 3), (2, 5, 47, 3)]),
    "length below zero": ([40, 20], [40, -20], None, 2, [(0, 0, 39, 1)]),
    "length below zero, no tokens": ([40, 20], [40, -1], [0, 2, 2], 2, [(0, 0, 38, 2)]),
    "length past the table": ([40, 20], [40, 49], None, 2, [(0, 0, 39, 1)]),
    "length past the table, no tokens": ([40, 20], [40, 49], [0, 2, 2], 2, [(0, 0, 38, 2)]),
    "largest numbers": ([40, 20], [40, (1 << 31) - 1], [0, 1, (1 << 31) - 1], 2, [(0, 0, 39, 1)]),
    "smallest numbers": ([40, 20], [-(1 << 31), 20], [-(1 << 31), 1, 2], 2, [(1, 1, 19, 1)]),
    "the hundredth of many": ([20] * 120, [20] * 99 + [-1] + [20] * 20, [min(i, 3) for i in range(121)], 3,
                              [(0, 0, 19, 1), (1, 1, 19, 1), (2, 2, 19, 1)]),
}


@pytest.mark.parametrize("queries", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_reported_and_not_written(case, queries):
    kv, lens, cu, T, written = CASES[case]
    cache = Cache(kv, HKV, S, D, BF, seed=3)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(T, HKV, D, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(T, 4, D, generator=g).to(BF).cuda() if queries else None
    want_k, want_v = cache.k.clone(), cache.v.clone()
    for b, row, pos, n in written:
        for i in range(n):
            page, slot = cache.table[b, (pos + i) // S].item(), (pos + i) % S
            want_k[page, :, slot], want_v[page, :, slot] = k[row + i], v[row + i]
    fa2.append_paged(k, v, cache.k, cache.v, cache.table, ints(lens), cu_q=ints(cu), q=q)
    torch.cuda.synchronize()
    status = fa2.fa2_device_status(None, reset=True)
    assert status == (fa2.FA2_OK if case == "in order" else fa2.FA2_ERR_PAGE)
    assert same(cache.k, want_k) and same(cache.v, want_v)


def test_many_blocks_report_once_and_in_graphs():
    """More tokens than a block takes, replayed after the offsets went wrong and right again."""
    n = [300, 500]
    cache = Cache(n, HKV, S, D, BF, seed=5)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(700, HKV, D, generator=g).to(BF).cuda() for _ in range(2))
    cu = ints([0, 300, 700])
    graph = torch.cuda.CUDAGraph()
    fa2.append_paged(k, v, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    torch.cuda.synchronize()
    good = cache.k.clone()
    with torch.cuda.graph(graph):
        fa2.append_paged(k, v, cache.k, cache.v, cache.table, cache.lens, cu_q=cu)
    for offsets, code in (([0, 300, 800], fa2.FA2_ERR_PAGE), ([0, 300, 700], fa2.FA2_OK)):
        cu.copy_(ints(offsets))
        graph.replay()
        torch.cuda.synchronize()
        assert fa2.fa2_device_status(None, reset=True) == code
        assert same(cache.k, good)

"""Reserving, forking, freeing, compacting and copying the pages of a cache,
against a model of it in Python."""
import random

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import release_memory

pytestmark = pytest.mark.gpu


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


class Model:
    """The same state and rules, one page at a time; a page's content is a number."""

    def __init__(self, B, M, P, S, planes=2):
        self.M, self.S, self.P = M, S, P
        self.rows, self.lens = [[] for _ in range(B)], [0] * B
        self.refs, self.content = [0] * P, [1000 + p for p in range(P)]
        self.table = torch.full((B, M + 3), -1, dtype=torch.int32, device="cuda")[:, :M]   # rows further apart
        self.d_lens, self.d_refs = ints(self.lens), ints(self.refs)
        self.pool = torch.empty((planes, P, 2, S, 8), dtype=torch.int32, device="cuda")
        self.pool[:] = ints(self.content)[None, :, None, None, None]
        self.pool[1:] += 100000

    def lowest(self, n):
        return [p for p in range(self.P) if self.refs[p] == 0][:n]

    def reserve(self, add):
        grow = [-(-(n + max(a, 0)) // self.S) - -(-n // self.S) for n, a in zip(self.lens, add)]
        fresh = self.lowest(sum(grow))
        wide = any(-(-(n + max(a, 0)) // self.S) > self.M for n, a in zip(self.lens, add))
        missing = -1 if wide else sum(grow) - len(fresh)
        if missing == 0:
            for b, (n, g) in enumerate(zip(add, grow)):
                for _ in range(g):
                    self.refs[fresh[0]] = 1
                    self.rows[b].append(fresh.pop(0))
                self.lens[b] += max(n, 0)
        got = fa2.pages_reserve(self.table, self.d_lens, self.d_refs, ints(add), self.S)
        assert got.item() == missing
        self.check()

    def fork(self, src, dst, bad=False):
        pairs, taken = [], set()
        for s, d in zip(src, dst):
            if 0 <= s < len(self.rows) and 0 <= d < len(self.rows) and not self.lens[d] and d not in taken:
                pairs.append((s, d))
                taken.add(d)
        part = [s for s, _ in pairs if self.lens[s] % self.S]
        fresh = self.lowest(len(part))
        missing = len(part) - len(fresh)
        if missing == 0:
            old_rows, old_lens = [list(r) for r in self.rows], list(self.lens)
            for s, d in pairs:
                full = old_lens[s] // self.S
                self.rows[d] = old_rows[s][:full]
                for p in self.rows[d]:
                    self.refs[p] += 1
                if old_lens[s] % self.S:
                    p = fresh.pop(0)
                    self.refs[p] = 1
                    self.content[p] = self.content[old_rows[s][full]]
                    self.rows[d].append(p)
                self.lens[d] = old_lens[s]
        got = fa2.pages_fork(self.table, self.d_lens, self.d_refs, ints(src), ints(dst), self.pool)
        assert got.item() == missing
        assert status() == (fa2.FA2_ERR_PAGE if bad else fa2.FA2_OK)
        self.check()

    def free(self, seqs):
        for b in set(seqs):
            for p in self.rows[b]:
                self.refs[p] -= 1
            self.rows[b], self.lens[b] = [], 0
        fa2.pages_free(self.table, self.d_lens, self.d_refs, ints(seqs))
        self.check()

    def compact(self):
        used = [p for p in range(self.P) if self.refs[p]]
        n = len(used)
        moved = [p if self.refs[p] else -1 for p in range(self.P)]
        holes = [p for p in range(n) if not self.refs[p]]
        for p, h in zip([p for p in used if p >= n], holes):
            moved[p] = h
            self.content[h] = self.content[p]
            self.refs[h], self.refs[p] = self.refs[p], 0
        self.rows = [[moved[p] for p in r] for r in self.rows]
        got = fa2.pages_compact(self.table, self.d_lens, self.d_refs, self.pool)
        assert got.tolist() == moved
        self.check()

    def check(self):
        assert self.d_lens.tolist() == self.lens
        assert self.d_refs.tolist() == self.refs
        assert self.table.tolist() == [r + [-1] * (self.M - len(r)) for r in self.rows]
        named = sorted({p for r in self.rows for p in r})
        want = ints([self.content[p] for p in named])[:, None, None, None]
        assert (self.pool[0][named] == want).all() and (self.pool[1:, named] == want[None] + 100000).all()


@pytest.mark.parametrize("S,P,B", [(16, 40, 5), (64, 300, 9), (1024, 20, 3), (16, 3000, 60)])
@pytest.mark.parametrize("seed", [0, 1])
def test_random_histories(S, P, B, seed):
    rng = random.Random(100 * seed + S + P)
    m = Model(B, max(4, 2 * P // B), P, S)
    for _ in range(25):
        what = rng.choice(["reserve", "reserve", "reserve", "fork", "free", "compact"])
        if what == "reserve":
            m.reserve([rng.choice([0, 1, S - 1, S, rng.randint(0, 3 * S)]) for _ in range(B)])
        elif what == "free":
            m.free([rng.randrange(B) for _ in range(rng.randint(1, 3))])     # the same one twice at times
        elif what == "fork":
            empty = [b for b in range(B) if not m.lens[b]]
            dst = rng.sample(empty, rng.randint(0, len(empty)))
            m.fork([rng.randrange(B) for _ in dst], dst)
        else:
            m.compact()
    assert status() == fa2.FA2_OK


def test_all_or_nothing():
    m = Model(3, 4, 6, 16)
    m.reserve([40, 17, 0])                # three pages and two: one is left
    m.reserve([0, 0, 17])                 # two lack one
    m.reserve([0, 0, 65])                 # more than a row holds
    m.reserve([8, -5, 3])                 # 48 and 3: the last page
    m.fork([1], [2], bad=True)            # not empty
    m.free([2])
    m.reserve([16, 0, 0])
    m.fork([1], [2])                      # its part needs a page, none is left
    m.free([0, 0])
    m.fork([1, 1, 1, 9, 1, -1], [2, 2, 0, 0, 7, 0], bad=True)   # twice the same, and indices outside
    m.compact()


def test_forks_of_this_call_are_not_sources():
    m = Model(4, 4, 20, 16)
    m.reserve([20, 0, 0, 0])
    m.fork([0, 1, 3], [1, 2, 3])          # 1 was empty before the call, and so is 2; 3 is its own copy
    m.fork([1, 1], [2, 3])
    m.free([0, 1])
    m.compact()


def test_many_pages_and_many_sequences():
    m = Model(1500, 40, 70000, 16, planes=1)
    rng = random.Random(3)
    m.reserve([rng.randint(0, 500) for _ in range(1500)])
    m.free(list(range(0, 1500, 2)))
    m.fork(list(range(1, 1500, 2)), list(range(0, 1500, 2)))
    m.compact()
    m.reserve([1] * 1500)


def test_copy_takes_the_last_pair_and_refuses_chains():
    P = 50
    pool = torch.arange(P, device="cuda", dtype=torch.int32)[:, None, None, None].expand(P, 2, 16, 4).contiguous()
    other = pool + 1000
    fa2.pages_copy([pool, other], ints([1, 2, 3, 7]), ints([10, 11, 10, 7]))
    want = list(range(P))
    want[10], want[11] = 3, 2
    assert pool[:, 0, 0, 0].tolist() == want and other[:, 1, 15, 3].tolist() == [w + 1000 for w in want]
    assert status() == fa2.FA2_OK
    fa2.pages_copy(pool, ints([20, 5, 6, 50, -1]), ints([21, 20, 22, 3, 4]))   # 20 is written by the second pair
    want[20], want[22] = 5, 6
    assert pool[:, 0, 0, 0].tolist() == want
    assert status() == fa2.FA2_ERR_PAGE


@pytest.mark.parametrize("shape", [(3, 1, 16, 8), (40, 3, 16, 64), (9, 8, 64, 128), (5, 2, 1024, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_copy_sizes_and_planes(shape, dtype):
    """Pages of odd numbers of chunks, in planes with gaps between the pages, with
    slots before heads, and in several leading dimensions."""
    P = shape[0]
    full = torch.randn((2, 3, P, 2) + shape[1:], generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    pool = full[:, :, :, 0]                      # every other page of the memory
    want = full.clone()
    src, dst = [0, 2], [1, 0][:1] + [P - 1]
    src, dst = ([0], [1]) if P == 3 else (src, dst)
    want[:, :, dst, 0] = full[:, :, src, 0]
    fa2.pages_copy(pool, ints(src), ints(dst))
    assert torch.equal(full, want)
    swapped = full[0, 0, :, 1].contiguous().transpose(1, 2)
    fa2.pages_copy(swapped, ints([0]), ints([1]))
    assert torch.equal(swapped[1], swapped[0])


def test_captured_reserve_and_fork():
    m = Model(4, 6, 30, 16)
    m.reserve([20, 5, 0, 0])
    table, lens, refs, pool = m.table.clone(), m.d_lens.clone(), m.d_refs.clone(), m.pool.clone()
    add, src, dst = ints([1, 12, 0, 0]), ints([0, 1]), ints([2, 3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = fa2.pages_fork(table, lens, refs, src, dst, pool)
        second = fa2.pages_reserve(table, lens, refs, add, 16)
    assert lens.tolist() == [20, 5, 0, 0]
    graph.replay()
    m.fork([0, 1], [2, 3])
    m.reserve([1, 12, 0, 0])
    assert first.item() == 0 and second.item() == 0
    assert torch.equal(table, m.table) and torch.equal(lens, m.d_lens) and torch.equal(refs, m.d_refs)
    assert torch.equal(pool, m.pool)


def test_freed_twice_is_reported():
    m = Model(2, 4, 8, 16)
    m.reserve([16, 0])
    m.d_refs.zero_()
    fa2.pages_free(m.table, m.d_lens, m.d_refs, ints([0]))
    assert status() == fa2.FA2_ERR_PAGE
    assert m.d_refs.tolist() == [0] * 8
    fa2.pages_free(m.table, m.d_lens, m.d_refs, ints([5]))
    assert status() == fa2.FA2_ERR_PAGE

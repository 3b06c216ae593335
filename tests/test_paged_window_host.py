"""The paged window and prefix entry points refuse bad arguments on the host; their schedule's closed forms in Python."""
import ctypes
import random

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from exact_attention_17_gb300 import paged
from test_paged_host import BAD_CACHES, cache


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return fa2.library()


def window(c, Q=16, qt=256, qh=64, O=16, LSE=16, cu=None, T=2, Hq=4, w=5, k=0, scale=0.125,
           o_dtype=fa2.FA2_DTYPE_BF16, ws=256, size=1 << 30):
    return fa2.library().fa2_forward_paged_window(None if c is None else ctypes.byref(c), Q, qt, qh, O, LSE, cu, T, Hq, w,
                                                  k, scale, o_dtype, ws, size, None)


def prefix(c, Q=16, qt=256, qh=64, O=16, LSE=16, cu=None, T=2, Hq=4, cg=16, pl=16, groups=1, scale=0.125,
           o_dtype=fa2.FA2_DTYPE_BF16, ws=256, size=1 << 30):
    return fa2.library().fa2_forward_paged_prefix(None if c is None else ctypes.byref(c), Q, qt, qh, O, LSE, cu, T, Hq, cg,
                                                  pl, groups, 1, scale, o_dtype, ws, size, None)


@pytest.mark.parametrize("call", [window, prefix])
def test_common_refusals(call):
    for bad, code in BAD_CACHES:
        assert call(cache(**bad)) == getattr(fa2, "FA2_ERR_" + code), bad
    c = cache()
    assert call(None) == fa2.FA2_ERR_NULL
    assert call(c, T=0, Q=None) == fa2.FA2_OK
    assert call(c, Hq=0) == fa2.FA2_OK
    assert call(cache(B=0)) == fa2.FA2_OK
    for bad in (dict(T=-1), dict(Hq=-4), dict(Hq=3), dict(Hq=258), dict(T=3), dict(qt=32), dict(qh=32)):
        assert call(c, **bad) == fa2.FA2_ERR_SHAPE, bad
    for dt in (fa2.FA2_DTYPE_FP16, 7):
        assert call(c, o_dtype=dt) == fa2.FA2_ERR_DTYPE
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert call(c, scale=s) == fa2.FA2_ERR_SCALE
    for name in ("Q", "O", "LSE", "ws"):
        assert call(c, **{name: None}) == fa2.FA2_ERR_NULL
    for name, value in (("Q", 8), ("O", 8), ("LSE", 2), ("ws", 128), ("cu", 2), ("qt", 260), ("qh", 68)):
        assert call(c, **{name: value}) == fa2.FA2_ERR_ALIGN, name


def test_own_refusals():
    c = cache()
    for bad in (dict(w=0), dict(w=-1), dict(k=-1)):
        assert window(c, **bad) == fa2.FA2_ERR_SHAPE, bad
    for bad in (dict(groups=-1), dict(groups=3)):
        assert prefix(c, **bad) == fa2.FA2_ERR_SHAPE, bad
    for bad in (dict(cg=None), dict(pl=None)):
        assert prefix(c, **bad) == fa2.FA2_ERR_NULL, bad
    for bad in (dict(cg=2), dict(pl=2)):
        assert prefix(c, **bad) == fa2.FA2_ERR_ALIGN, bad
    f = fa2.library().fa2_forward_paged_prefix_workspace_bytes
    for bad in ((0, 1, 4, 8, 2, 64, 0), (2, 0, 2, 8, 2, 64, 0), (2, 1, 0, 8, 2, 64, 0), (2, 1, 2, 7, 2, 64, 0),
                (2, 1, 2, 8, 2, 96, 0), (2, 1, 2, 258, 2, 64, 0)):
        assert f(*bad) == 0


@pytest.fixture(params=["binding", "ctypes"])
def way(request, monkeypatch):
    if paged.torch is None:
        paged._load()
    if request.param == "ctypes":
        monkeypatch.setattr(paged, "_fast", None)


def test_python_calls_check_their_tensors(way):
    k, q = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        fa2.forward_paged_window(q, k, k, i32(2, 3), i32(2), 5)
    with pytest.raises(ValueError, match="CUDA"):
        fa2.forward_paged_prefix(q, k, k, i32(2, 3), i32(2), i32(2), i32(1))
    for bad in ((0, 0), (5, -1)):
        with pytest.raises(ValueError, match="window"):
            fa2.forward_paged_window(q, k, k, i32(2, 3), i32(2), *bad)


TILE = 128


def tiles_of(keys):
    return -(-keys // TILE)


def test_lists_and_costs():
    """The kernel's list of a block (pages, or tiles of larger pages, with sinks, then those of its windows) holds every
    key that a row sees; the closed form of the blocks' costs is the sum of theirs, and a block's cost reaches its last
    tile."""
    rng = random.Random(5)
    for _ in range(3000):
        block, unit = rng.choice([1, 4, 18, 32, 128, 256]), rng.choice([16, 32, 64, 128])
        window = rng.choice([1, 5, 127, 128, 129, rng.randint(1, 3000)])
        sinks = rng.choice([0, 1, 128, 130, rng.randint(0, 600)])
        kv, q = rng.randint(0, 4000), rng.randint(1, 1200)
        fixed = rng.choice([256, 512])
        blocks = -(-q // block)
        most = (-(-sinks // unit) + (block - 1 + window + 2 * unit - 2) // unit) * unit

        def keys(i):
            return max(1, max(0, min(kv, kv - q + min((i + 1) * block, q))))

        for i in rng.sample(range(blocks), min(blocks, 4)):
            first, last = kv - q + i * block, kv - q + min((i + 1) * block, q) - 1
            lo = max(0, first - window + 1) // unit * unit
            sink_keys = min(-(-sinks // unit) * unit, lo)
            skip = lo - sink_keys
            kept = max(0, min(kv, last + 1))
            listed = [x if x < sink_keys else x + skip for x in range(max(0, kept - skip))]
            assert listed == sorted(set(listed)) and len(listed) <= most
            every = set(listed)
            for row in {first, last, rng.randint(first, last)}:
                if row >= 0:
                    assert set(range(max(0, row - window + 1), row + 1)) <= every
                    assert set(range(min(sinks, row + 1))) <= every
            tiles = tiles_of(keys(i) - skip)
            assert 1 <= tiles <= tiles_of(min(keys(i), most)) and (kept == 0 or tiles == tiles_of(len(listed)))

        # cost_before
        for i in rng.sample(range(blocks + 1), min(blocks + 1, 4)):
            want = sum(fixed + min(keys(k), most) for k in range(i))
            if i == 0:
                got = 0
            else:
                full = i - 1 if i == blocks else i
                lead = kv - q
                none = 0 if lead >= 0 else min(full, -lead // block)
                n = full - none
                got = none
                below = 0 if lead > most else (most - lead) // block
                capped = max(0, min(n, full - below))
                got += capped * most
                n -= capped
                got += n * (lead + none * block) + block * (n * (n + 1) // 2) + i * fixed
                if i == blocks:
                    got += max(1, min(kv, most))
            assert got == want, (block, window, sinks, kv, q, i)


def test_entries_of_blocks():
    """Blocks of all sequences have entries of their own (the parts that the joining kernel looks up)."""
    rng = random.Random(6)
    for _ in range(500):
        block, B = rng.choice([1, 2, 5, 32, 128]), rng.randint(1, 30)
        lens = [rng.choice([0, 1, rng.randint(0, 300)]) for _ in range(B)]
        T, q0, seen = sum(lens) + rng.randint(0, 5), 0, []
        for b, n in enumerate(lens):
            seen += [q0 // block + i + b for i in range(-(-n // block))]
            q0 += n
        assert len(seen) == len(set(seen)) and all(0 <= x < T // block + B + 1 for x in seen)

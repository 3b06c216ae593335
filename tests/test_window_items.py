"""The items of the windowed gradients, restated in Python: how a block of the grid finds its key block, head and
query tiles when heads run in groups, the last of them shorter, and key blocks are cut.  Every query tile of every key
block and query head is some item's exactly once, items of one key block have workspace slots of their own, and the
kernel behind adds up exactly those."""
import ctypes

import pytest

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild

TILE = 128


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return fa2.library()


def tiles(n):
    return -(-n // TILE)


SHAPES = [
    # B, H, Hkv, Nq, Nk, d, window, sinks
    (2, 48, 6, 600, 600, 128, 300, 0),
    (1, 56, 7, 600, 600, 128, 300, 4),
    (1, 40, 5, 600, 600, 128, 300, 200),
    (3, 76, 19, 300, 300, 128, 100, 4),
    (1, 56, 7, 500, 200, 128, 300, 130),
    (1, 56, 7, 200, 700, 128, 150, 0),
    (1, 56, 7, 200, 700, 128, 150, 690),
    (4, 16, 4, 4096, 4096, 128, 1024, 4),
    (3, 16, 4, 4096, 4096, 128, 1024, 4),
    (1, 24, 6, 8192, 8192, 128, 2048, 4),
    (1, 2, 1, 1, 300, 128, 5, 2),
    (1, 3, 3, 1000, 77, 64, 30, 0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_every_tile_once(shape):
    B, H, Hkv, Nq, Nk, d, window, sinks = shape
    out = (ctypes.c_int * 4)()
    assert fa2.library().fa2_check_window_plan(*shape, 152, out) == fa2.FA2_OK
    _, group, parts, sink_parts = out
    BH, shared, window, sinks = B * Hkv, H // Hkv, min(window, Nq), min(sinks, Nk)
    key_blocks, sink_blocks, q_tiles = tiles(Nk), tiles(sinks), tiles(Nq)
    assert 1 <= group <= BH
    row = min((126 + window) // TILE + 1, q_tiles)
    chunk, sink_chunk = -(-row * shared // parts), -(-q_tiles * shared // sink_parts)
    items = BH * (sink_blocks * sink_parts + (key_blocks - sink_blocks) * parts)
    sink_slots = BH * sink_blocks * sink_parts
    per_head = sink_blocks * sink_parts + (key_blocks - sink_blocks) * parts
    taken, slots = {}, {}
    for x in range(items):
        g0 = x // (group * per_head) * group
        heads, inside = min(group, BH - g0), x - g0 * per_head
        sink_items = heads * sink_blocks * sink_parts
        with_sinks = inside < sink_items
        n = sink_parts if with_sinks else parts
        y, part = divmod(inside - (0 if with_sinks else sink_items), n)
        jb, bh = y // heads, g0 + y % heads
        slot = (jb * BH + bh) * n + part + (0 if with_sinks else sink_slots) if n > 1 else None
        jb += 0 if with_sinks else sink_blocks
        assert 0 <= bh < BH and 0 <= jb < key_blocks
        i0 = min(jb, q_tiles)
        last = min(jb * TILE + TILE - 1, Nk - 1) + window - 1
        end = q_tiles if with_sinks else min(q_tiles, last // TILE + 1)
        rows, size = max(0, end - i0), sink_chunk if with_sinks else chunk
        first = part * size
        for t in range(first, first + max(0, min(size, rows * shared - first))):
            where = jb, bh * shared + t // rows, i0 + t % rows
            assert where not in taken
            taken[where] = x
        if slot is not None:
            assert slot not in slots
            slots[slot] = jb, bh
    # every tile with a (query, key) pair that is seen
    for jb in range(key_blocks):
        k0, k1 = jb * TILE, min(jb * TILE + TILE, Nk) - 1
        seen = {i for i in range(q_tiles)
                if any(k0 <= q and (k0 < sinks or q - min(k1, q) < window) for q in range(i * TILE, min(Nq, i * TILE + TILE)))}
        for h in range(BH * shared):
            assert all((jb, h, i) in taken for i in seen)
    # what the kernel behind reads for a block
    held = items if parts > 1 else sink_slots if sink_parts > 1 else 0
    for jb in range(key_blocks):
        for bh in range(BH):
            y, with_sinks = jb * BH + bh, jb < sink_blocks
            n = sink_parts if with_sinks else parts
            if n == 1:
                continue
            base = y * n if with_sinks else sink_slots + (y - BH * sink_blocks) * n
            assert all(slots[base + i] == (jb, bh) and base + i < held for i in range(n))


def test_groups_are_equal_where_they_hold_four_heads():
    def group(*shape):
        out = (ctypes.c_int * 4)()
        assert fa2.library().fa2_check_window_plan(*shape, 152, out) == fa2.FA2_OK
        return out[1]

    assert group(4, 16, 4, 4096, 4096, 128, 1024, 4) == 8        # 16 heads, of which 11 fit
    assert group(3, 16, 4, 4096, 4096, 128, 1024, 4) == 6        # 12
    assert group(1, 24, 6, 8192, 8192, 128, 2048, 4) == 5        # 6, of which 5 fit: three each are too few
    assert group(1, 40, 5, 600, 600, 128, 300, 0) == 4           # 5, of which none fit: four all the same
    assert group(1, 56, 7, 600, 600, 128, 300, 0) == 4
    assert group(1, 4, 2, 600, 600, 128, 300, 0) == 2            # all of them

"""The schedule of the paged attention kernel, restated in Python.

Each CTA of the kernel finds its work from lengths on the device.  The list of
all items (sequence, key/value head, block of tokens) has closed-form costs; with
equal ranges a CTA takes the tiles between two positions of the list, without
them whole items in an order of their own, long ones cut.  Restated here with
the kernel's arithmetic and checked on random batches: every tile of every item
is taken once, parts of one item lie in workspace slots of their own, and the
merge reads exactly those, in the order of the keys.
"""
import random

import pytest

KEYS = 128   # keys of a tile


def tiles_of(keys):
    return -(-keys // KEYS)


def kept(causal, kv, q, tok):
    return max(0, min(kv, kv - q + tok + 1)) if causal else kv


class Batch:
    def __init__(self, rng, long_items=False):
        self.causal = rng.random() < 0.8
        self.heads = rng.choice([1, 2, 3, 40])
        self.block = rng.choice([1, 4, 18, 24, 48, 128, 256])
        n = rng.choice([1, 2, 5, 40])
        most = 1200 if self.heads < 40 else 60
        self.q = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(n)]
        self.kv = [rng.choice([0, rng.randint(0, 20000 if long_items else 5000)]) for _ in range(n)]
        self.blocks = [-(-x // self.block) for x in self.q]
        self.ctas = rng.choice([4, 152, 304])
        self.min_tiles = 1
        self.per_item = rng.choice([256, 512])   # an item's fixed cost in keys

    def keys(self, b, i):
        return max(1, kept(self.causal, self.kv[b], self.q[b], min((i + 1) * self.block, self.q[b]) - 1))

    def cost_before(self, b, i):
        """Cost of the blocks 0 .. i-1, as the kernel computes it."""
        if i == 0:
            return 0
        full = i - 1 if i == self.blocks[b] else i
        if self.causal:
            lead = self.kv[b] - self.q[b]
            none = 0 if lead >= 0 else min(full, -lead // self.block)
            n = full - none
            keys = none + n * (lead + none * self.block) + self.block * (n * (n + 1) // 2)
        else:
            keys = full * max(1, self.kv[b])
        keys += i * self.per_item
        return keys + (max(1, self.kv[b]) if i == self.blocks[b] else 0)

    def total(self):
        return sum(self.cost_before(b, self.blocks[b]) for b in range(len(self.q))) * self.heads

    def share(self):
        return max(int(self.total() * (1.0 / self.ctas)) + 2, self.min_tiles * KEYS + self.per_item)

    def find(self, pos):
        """[sequence, head, block, start of the item] that the position lies in."""
        start = 0
        for b, n in enumerate(self.blocks):
            each = self.cost_before(b, n)
            if pos >= start + each * self.heads:
                start += each * self.heads
                continue
            head = (pos - start) // each
            start += head * each
            lo, left = 0, n
            while left > 1:   # 32 candidates at a time
                step = -(-left // 32)
                last = max(x for x in range(32)
                           if x * step < left and start + self.cost_before(b, lo + min(x * step, left)) <= pos)
                left, lo = min(step, left - last * step), lo + last * step
            return [b, head, lo, start + self.cost_before(b, lo)]
        raise AssertionError("position behind the list")

    def tile(self, item, pos):
        b, _, i, start = item
        keys = self.keys(b, i)
        x = pos - start - self.per_item
        if x <= 0:
            return 0
        return tiles_of(keys) if pos >= start + self.per_item + keys else min(tiles_of(keys), tiles_of(x))

    def walk(self, cta):
        """Segments (item, first tile, last tile, slot) of a range."""
        share, total = self.share(), self.total()
        lo, hi = cta * share, min((cta + 1) * share, total)
        if lo >= hi:
            return
        at = self.find(lo)
        while lo < hi:
            first, last = self.tile(at, lo), self.tile(at, hi)
            if first < last:
                whole = tiles_of(self.keys(at[0], at[2]))
                yield tuple(at[:3]), first, last, 2 * cta if first > 0 else 2 * cta + 1 if last < whole else -1
            at[3] += self.per_item + self.keys(at[0], at[2])
            lo = max(lo, at[3])
            at[2] += 1
            if at[2] == self.blocks[at[0]]:
                at[2] = 0
                at[1] += 1
                if at[1] == self.heads:
                    more = [b for b in range(at[0] + 1, len(self.q)) if self.blocks[b]]
                    if not more:
                        return
                    at[1], at[0] = 0, more[0]

    def merges(self):
        """(item, slots in the order of the keys) of each item that the merge kernel's CTAs find."""
        share, total = self.share(), self.total()
        for index in range(self.ctas - 1):
            pos = (index + 1) * share
            if pos >= total:
                continue
            at = self.find(pos)
            whole = tiles_of(self.keys(at[0], at[2]))
            t = self.tile(at, pos)
            if t == 0 or t == whole or self.tile(at, pos - share) > 0:
                continue
            parts, nxt = 2, pos + share
            while nxt < total and self.tile(at, nxt) < whole:
                parts, nxt = parts + 1, nxt + share
            yield tuple(at[:3]), [2 * index + 1] + [2 * (index + 1) + 2 * k for k in range(parts - 1)]


@pytest.mark.parametrize("seed", range(60))
def test_equal_ranges_cover_every_item_once(seed):
    rng = random.Random(seed)
    batch = Batch(rng)
    for b, n in enumerate(batch.blocks):
        for i in range(n + 1):
            assert batch.cost_before(b, i) == sum(batch.per_item + batch.keys(b, k) for k in range(i))
    if batch.total() == 0:
        return
    assert batch.share() * batch.ctas >= batch.total()
    cover, slots = {}, {}
    for cta in range(batch.ctas):
        for item, first, last, slot in batch.walk(cta):
            cover.setdefault(item, []).append((first, last, slot))
            if slot >= 0:
                assert slot < 2 * batch.ctas and slot not in slots
                slots[slot] = (item, first, last)
    assert len(cover) == sum(batch.blocks) * batch.heads
    cut = {}
    for item, parts in cover.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == tiles_of(batch.keys(item[0], item[2]))
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
        if len(parts) > 1:
            cut[item] = [slot for _, _, slot in parts]
        else:
            assert parts[0][2] == -1
    assert dict(batch.merges()) == cut


L2_BYTES = 64 << 20


@pytest.mark.parametrize("seed", range(40))
def test_whole_items_in_their_order(seed):
    """Items one by one: units and merged items are numbered without gaps, slots and counts stay in their bounds."""
    rng = random.Random(1000 + seed)
    batch = Batch(rng, long_items=True)
    d = 128
    tiles = [tiles_of(x) for x in batch.kv]
    total = sum(n * t for n, t in zip(batch.blocks, tiles)) * batch.heads
    per_unit = max(batch.min_tiles, -(-total // batch.ctas))
    splits = [max(1, -(-t // per_unit)) for t in tiles]
    units = [n * batch.heads * s for n, s in zip(batch.blocks, splits)]
    most_items = (sum(batch.q) // batch.block + min(len(batch.q), sum(batch.q))) * batch.heads
    assert sum(units) <= most_items + batch.ctas
    assert sum(u for u, s in zip(units, splits) if s > 1) <= 2 * batch.ctas
    assert sum(n * batch.heads for n, s in zip(batch.blocks, splits) if s > 1) <= batch.ctas

    def locate(index, items):
        before = slots = 0
        for b, (n, s) in enumerate(zip(batch.blocks, splits)):
            count = (n * batch.heads if s > 1 else 0) if items else n * batch.heads * s
            if before <= index < before + count:
                at = (index - before) * (s if items else 1)
                slot = slots + at
                group_heads = int(min(max(L2_BYTES // (max(batch.kv[b], 1) * d * 4), 1), batch.heads))
                group, at = divmod(at, group_heads * n * s)
                per_block = min(group_heads, batch.heads - group * group_heads) * s
                rank, at = divmod(at, per_block)
                head, split = divmod(at, s)
                return (b, group * group_heads + head, n - 1 - rank), split, slot
            before += count
            slots += n * batch.heads * s if s > 1 else 0
        return None

    seen, slot_of = set(), {}
    for index in range(sum(units)):
        item, split, slot = locate(index, False)
        assert (item, split) not in seen and item[1] < batch.heads and 0 <= item[2] < batch.blocks[item[0]]
        seen.add((item, split))
        if splits[item[0]] > 1:
            assert slot not in slot_of.values()
            slot_of[item, split] = slot
    assert locate(sum(units), False) is None and len(seen) == sum(units)
    merged = sum(n * batch.heads for n, s in zip(batch.blocks, splits) if s > 1)
    for index in range(merged):
        item, split, slot = locate(index, True)
        assert split == 0
        assert [slot_of.pop((item, k)) for k in range(splits[item[0]])] == list(range(slot, slot + splits[item[0]]))
    assert not slot_of and locate(merged, True) is None


@pytest.mark.parametrize("stages", [2, 4, 5, 8])
def test_last_copies_that_a_producer_waits_for(stages):
    """A barrier's phase is known by its parity: waiting for one that a later copy
    of the slot has superseded would never end.  The last `stages` copies are the
    last of their slots."""
    for copies in range(2, 60, 2):
        last = {}
        for i in range(copies):
            last[i % stages] = i
        assert sorted(last.values()) == list(range(max(0, copies - stages), copies))


@pytest.mark.parametrize("log2", range(4, 11))
def test_page_cursor_finds_every_page(log2):
    """32 table entries at a time: a tile's pages never straddle two chunks, from any first tile on."""
    pages_of_tile = KEYS >> min(log2, 7)
    for first_tile in range(0, 40, 7):
        chunk = (first_tile << 7) >> log2
        for tile in range(first_tile, first_tile + 200):
            first = (tile << 7) >> log2
            if first >= chunk + 32:
                chunk += 32
            assert chunk <= first and first + pages_of_tile <= chunk + 32

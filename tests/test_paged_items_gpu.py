"""The form of forward_paged that takes whole items from a counter (batches of many blocks), items cut among them.

A batch is many short chunks beside one over many keys: enough blocks for the form, and a sequence long
enough to be cut.  The counter, which the call keeps behind the partial results of its workspace, says
afterwards how many units there were; the form of equal ranges does not touch it.
"""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import Cache, offsets, release_memory
from test_paged_gpu import check, queries

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


def block_tokens(d, G, subs):
    """Tokens of a block: whole groups of eight rows as far as 128 rows hold them."""
    unit = 8 // math.gcd(G, 8)
    most = 128 // G
    box = unit if most >= unit else most
    return most // box * box * subs


CASES = [
    # dtype, d, Hq, Hkv, page, sub-tiles, tokens of a short chunk, the long sequence's tokens and keys, causal
    (BF, 128, 16, 4, 16, 2, 64, 50, 30000, True),
    (HF, 128, 8, 8, 64, 2, 300, 257, 9000, True),          # a second block, a chunk of a block and a bit
    (BF, 128, 12, 12, 32, 2, 256, 1, 20000, False),
    (HF, 64, 24, 8, 32, 2, 80, 33, 20000, True),           # three heads a group
    (BF, 64, 16, 16, 128, 2, 256, 300, 5000, False),
    (BF, 64, 32, 8, 16, 1, 20, 40, 9000, True),            # one sub-tile, two CTAs an SM
    (HF, 128, 32, 8, 16, 1, 24, 3, 7000, True),
    (HF, 128, 32, 8, 256, 1, 24, 3, 7000, False),
    (BF, 256, 16, 4, 64, 1, 32, 70, 12000, True),
    (HF, 256, 8, 8, 16, 1, 100, 128, 3000, False),
    (BF, 256, 14, 2, 128, 1, 16, 1, 20000, True),          # seven heads a group
]


def batch(case, sms):
    dtype, d, Hq, Hkv, S, subs, short, long_q, long_kv, causal = case
    G, ctas = Hq // Hkv, sms * (1 if subs == 2 or d == 256 else 2)
    block = block_tokens(d, G, subs)
    tokens = ((2 if d == 256 else 4) * ctas * block * 5 // 4) // Hkv     # a quarter more than the form asks for
    q_lens = [short - i % 3 for i in range(-(-tokens // (short - 1)))]
    kv = [n + (i * 61) % 150 for i, n in enumerate(q_lens)]
    kv[2] = q_lens[2] - 2                                                # rows without keys, when causal
    at = len(q_lens) // 3
    q_lens.insert(at, long_q)
    kv.insert(at, long_kv)
    q_lens.insert(at, 0)
    kv.insert(at, 70)
    T = sum(q_lens)
    assert T * G > 32 * len(kv) and (subs == 2) == (d != 256 and T * G > 128 * len(kv))
    items = sum(-(-n // block) for n in q_lens) * Hkv
    total = sum(-(-n // block) * -(-m // 128) for n, m in zip(q_lens, kv)) * Hkv
    share = -(-total // ctas)
    units = sum(-(-n // block) * max(1, -(-(-(-m // 128)) // share)) for n, m in zip(q_lens, kv)) * Hkv
    return q_lens, kv, items, units


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{str(c[0])[6:]}-d{c[1]}-h{c[2]}.{c[3]}-{c[5]}x{'c' if c[9] else 'n'}")
def test_matches_the_64_bit_form(case):
    dtype, d, Hq, Hkv, S, subs, short, long_q, long_kv, causal = case
    q_lens, kv, items, units = batch(case, torch.cuda.get_device_properties(0).multi_processor_count)
    cache = Cache(kv, Hkv, S, d, dtype, seed=d + Hq)
    q = queries(q_lens, Hq, d, dtype, seed=Hq)
    T, cu = sum(q_lens), offsets(q_lens)
    need = fa2.library().fa2_forward_paged_workspace_bytes(len(kv), T, Hq, Hkv, d, 1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    first = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu, causal=causal, workspace=ws)
    assert ws[need - 256:need - 252].view(torch.int32).item() == units > items     # this form, and items were cut
    check(*first, q, cache, q_lens, causal, 1 / math.sqrt(d))
    # 32-bit outputs; and who takes an item does not show
    for _ in range(2):
        o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=cu, causal=causal,
                                   out_dtype=torch.float32, workspace=ws)
        assert torch.equal(o.to(dtype), first[0]) and torch.equal(lse, first[1])
    check(o, lse, q, cache, q_lens, causal, 1 / math.sqrt(d), torch.float32)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_nothing_to_cut(d):
    """Chunks of one length and nothing longer: no item has parts, and the merge finds none."""
    Hq = Hkv = 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    block = block_tokens(d, 1, 1 if d == 256 else 2)
    n = -(-(2 if d == 256 else 4) * sms * 5 // (4 * Hkv))
    q_lens, kv = [block] * n, [block + 37] * n
    cache = Cache(kv, Hkv, 32, d, BF, seed=9)
    q = queries(q_lens, Hq, d, BF, seed=10)
    need = fa2.library().fa2_forward_paged_workspace_bytes(n, sum(q_lens), Hq, Hkv, d, 1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    o, lse = fa2.forward_paged(q, cache.k, cache.v, cache.table, cache.lens, cu_q=offsets(q_lens), workspace=ws)
    assert ws[need - 256:need - 252].view(torch.int32).item() == n * Hkv
    check(o, lse, q, cache, q_lens, True, 1 / math.sqrt(d))

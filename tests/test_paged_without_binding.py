"""The paged calls without the compiled binding: ctypes alone, the same checks, the same results."""
import os

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from exact_attention_17_gb300 import paged

BF = torch.bfloat16


@pytest.fixture
def without_binding(monkeypatch):
    libbuild.build()
    there = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: there(p) and p != libbuild.BINDING_PATH)
    for name in ("torch", "_lib", "_fast", "_codes", "_raw_stream"):
        monkeypatch.setattr(paged, name, None)


def test_arguments_are_checked(without_binding):
    k = torch.zeros(4, 2, 16, 64, dtype=BF)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(2, 4, 64, dtype=BF)
    calls = [lambda: fa2.forward_paged(q, k, k, i32(2, 3), i32(2)),
             lambda: fa2.append_paged(q[:, :2], q[:, :2], k, k, i32(2, 3), i32(2), q=q),
             lambda: fa2.rope(q, i32(2), torch.zeros(32, dtype=torch.float64)),
             lambda: fa2.pages_reserve(i32(2, 3), i32(2), i32(4), i32(2), 16),
             lambda: fa2.pages_fork(i32(2, 3), i32(2), i32(4), i32(1), i32(1), k),
             lambda: fa2.pages_free(i32(2, 3), i32(2), i32(4), i32(1)),
             lambda: fa2.pages_compact(i32(2, 3), i32(2), i32(4), k),
             lambda: fa2.pages_copy(k, i32(1), i32(1))]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert paged._fast is None


def step():
    """Room, append, attention, a fork, a copy, a compaction and a release; everything they leave."""
    d, Hq, Hkv, S = 64, 8, 2, 16
    g = torch.Generator().manual_seed(1)
    pool = torch.zeros((2, 32, Hkv, S, d), dtype=BF, device="cuda")
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, refs = ints([0, 0, 0]), ints([0] * 32)
    q, k, v = (torch.randn(45, h, d, generator=g).to(BF).cuda() for h in (Hq, Hkv, Hkv))
    freq = fa2.rope_inv_freq(d, device="cuda")
    cu = ints([0, 40, 45, 45])
    out = [fa2.pages_reserve(table, lens, refs, ints([40, 5, 0]), S)]
    out.append(fa2.append_paged(k, v, pool[0], pool[1], table, lens, cu, q=q, inv_freq=freq))
    out += fa2.forward_paged(out[-1], pool[0], pool[1], table, lens, cu_q=cu)
    out.append(fa2.rope(q, torch.arange(45, device="cuda"), freq))
    out.append(fa2.rope_backward(q, torch.arange(45, device="cuda"), freq))
    out.append(fa2.pages_fork(table, lens, refs, ints([0]), ints([2]), pool))
    fa2.pages_copy(pool, ints([0, 1]), ints([30, 31]))
    fa2.pages_free(table, lens, refs, ints([0]))
    out.append(fa2.pages_compact(table, lens, refs, pool))
    torch.cuda.synchronize()
    return out + [pool, table, lens, refs]


@pytest.mark.gpu
def test_the_same_results(without_binding, monkeypatch):
    got = step()
    assert paged._fast is None
    monkeypatch.undo()
    paged._load()
    assert paged._fast is not None
    for a, b in zip(got, step()):
        assert torch.equal(a, b)

"""Attention with shared prefixes and with windows directly between writers of what it reads, without a wait anywhere, on
one stream and on two at once: the same bits as with the device idle before every call."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, Cache, offsets, release_memory
from test_paged_window_gpu import BF, HF, ints, normal, share, status

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


class Server:
    """Steps that write the last positions of every sequence, attend, and write NaN over what was read."""

    def __init__(self, dtype, d, Hq, Hkv, S, samples, prompt, new, seed, steps=6):
        kv = [prompt + 7 * i % 90 + new for i in range(samples)]
        self.cache = Cache(kv, Hkv, S, d, dtype, seed=seed)
        share(self.cache, [0, samples // 2, samples], [prompt, prompt - S])
        self.prefix = ints([0, samples // 2, samples]), ints([prompt, prompt - S])
        self.cu = None if new == 1 else offsets([new] * samples)
        T = samples * new
        self.steps = [[normal((T, h, d), dtype, 1000 * seed + 3 * i + x) for x, h in enumerate((Hq, Hkv, Hkv))]
                      for i in range(steps)]
        self.nan = torch.full((T, Hkv, d), float("nan"), dtype=dtype, device="cuda")
        self.q = torch.empty_like(self.steps[0][0])
        self.spread = max(v.abs().max().item() for v in self.cache.values) + 5

    def append(self, k, v):
        c = self.cache
        fa2.append_paged(k, v, c.k, c.v, c.table, c.lens, cu_q=self.cu)

    def step(self, i, which):
        c, (q, k, v) = self.cache, self.steps[i]
        at = (self.q, c.k, c.v, c.table, c.lens)
        self.q.copy_(q)
        self.append(k, v)
        if which == "prefix":
            out = fa2.forward_paged_prefix(*at, *self.prefix, cu_q=self.cu)
        elif which == "window":
            out = fa2.forward_paged_window(*at, 500, 4, cu_q=self.cu)
        else:
            out = fa2.forward_paged(*at, cu_q=self.cu)
        self.append(self.nan, self.nan)
        self.q.fill_(float("nan"))
        return out

    def idle(self, which):
        out = []
        for i in range(len(self.steps)):
            torch.cuda.synchronize()
            out.append(self.step(i, which))
        torch.cuda.synchronize()
        return out


SERVERS = [
    # dtype, d, Hq, Hkv, page, sequences, shared tokens, new tokens
    (BF, 128, 32, 8, 16, 32, 4096, 1),
    (HF, 64, 16, 4, 32, 12, 6016, 5),
    (BF, 256, 8, 2, 16, 6, 2048, 70),
    (BF, 128, 16, 4, 64, 4, 4032, 600),
]
IDS = [f"{str(c[0])[6:]}-d{c[1]}-b{c[5]}-p{c[6]}-n{c[7]}" for c in SERVERS]


@pytest.mark.parametrize("which", ["prefix", "window"])
@pytest.mark.parametrize("case", SERVERS, ids=IDS)
def test_between_writers(case, which):
    server = Server(*case, seed=1)
    want = server.idle(which)
    for _ in range(3):
        got = [server.step(i, which) for i in range(len(server.steps))]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    if which == "prefix":
        for (o, lse), (ref, ref_lse) in zip(want, server.idle("plain")):
            # each side rounds P (relative u of sum p |v| <= max |v|) and O
            u = EPS[case[0]]
            assert ((o.double() - ref.double()).abs() <= 2.5 * u * server.spread + 2 * u * ref.double().abs()).all()
            assert (lse - ref_lse).abs().max() <= 1e-4
    assert status() == fa2.FA2_OK


@pytest.mark.parametrize("case", SERVERS, ids=IDS)
def test_two_streams_at_once(case):
    servers, streams = [Server(*case, seed=s) for s in (2, 3)], [torch.cuda.Stream() for _ in range(2)]
    kinds = [("prefix", "prefix"), ("prefix", "window")]
    want = [{w: s.idle(w) for w in ("prefix", "window")} for s in servers]
    for kind in kinds:
        torch.cuda.synchronize()
        got = [[], []]
        for i in range(len(servers[0].steps)):
            for server, stream, which, out in zip(servers, streams, kind, got):
                with torch.cuda.stream(stream):
                    out.append(server.step(i, which))
        torch.cuda.synchronize()
        for which, out, ref in zip(kind, got, want):
            for a, b in zip(out, ref[which]):
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert status() == fa2.FA2_OK

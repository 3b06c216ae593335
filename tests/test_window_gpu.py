"""Attention with a window and sinks, and its gradients, against 64-bit forms."""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, release_memory
from window_reference import backward, forward, seen

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


def normal(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def close(y, ref, bound, name=""):
    worst = ((y.double() - ref).abs() / (bound + 1e-30)).max() if y.numel() else 0.0
    assert worst <= 1.0, f"{name} off by {worst:.3f} of the bound"


def inputs(dtype, B, H, Hkv, Nq, Nk, d, std=1.0):
    return (normal((B, H, Nq, d), dtype, 1, std), normal((B, Hkv, Nk, d), dtype, 2, std),
            normal((B, Hkv, Nk, d), dtype, 3))


def check_forward(q, k, v, window, sinks, out_dtype=F32):
    d = q.shape[-1]
    scale = 1.0 / math.sqrt(d)
    o, lse = fa2.forward_window(q, k, v, window, sinks, out_dtype=out_dtype)
    assert o.dtype is out_dtype and lse.dtype is F32
    ref, ref_lse, bO, bL, _, _ = forward(q, k, v, seen(q.shape[2], k.shape[2], window, sinks), scale,
                                         EPS[out_dtype])
    close(o, ref, bO, "O")
    none = ref_lse == -math.inf
    assert torch.equal(lse == -math.inf, none) and (o[none] == 0).all()
    close(lse[~none], ref_lse[~none], bL[~none], "LSE")
    return o, lse


FORWARD = [
    # dtype, B, H, Hkv, Nq, Nk, d, window, sinks
    (BF, 1, 1, 1, 1, 1, 64, 1, 0),
    (BF, 1, 2, 1, 1, 300, 128, 5, 2),
    (HF, 1, 2, 2, 130, 130, 64, 1, 0),              # each query its own key
    (BF, 2, 4, 2, 300, 300, 128, 64, 0),
    (BF, 1, 3, 1, 500, 500, 64, 127, 1),
    (HF, 1, 8, 2, 513, 513, 128, 128, 4),
    (BF, 1, 2, 2, 700, 700, 256, 129, 3),
    (BF, 1, 2, 1, 1000, 1000, 64, 200, 130),        # sinks over a tile's end
    (BF, 1, 2, 2, 900, 900, 128, 100, 300),
    (HF, 1, 2, 2, 640, 640, 128, 5000, 0),          # the window holds everything
    (BF, 1, 2, 2, 640, 640, 64, 10, 5000),          # so do the sinks
    (BF, 1, 2, 1, 700, 200, 128, 150, 0),           # late rows without a key
    (BF, 1, 2, 1, 700, 200, 256, 150, 2),
    (HF, 1, 1, 1, 1000, 77, 64, 30, 0),             # whole blocks without a key
    (BF, 1, 2, 2, 200, 900, 128, 64, 4),            # more keys than queries
    (BF, 2, 40, 8, 1024, 1024, 64, 300, 4),         # two sub-tiles a CTA
    (HF, 2, 40, 40, 1100, 1100, 128, 128, 0),
    (BF, 2, 40, 10, 1030, 600, 128, 250, 0),
]
IDS = [f"{str(c[0])[6:]}-{c[1]}x{c[2]}.{c[3]}x{c[4]}.{c[5]}x{c[6]}-w{c[7]}-s{c[8]}" for c in FORWARD]


@pytest.mark.parametrize("case", FORWARD, ids=IDS)
def test_forward(case):
    dtype, B, H, Hkv, Nq, Nk, d, window, sinks = case
    q, k, v = inputs(dtype, B, H, Hkv, Nq, Nk, d)
    check_forward(q, k, v, window, sinks)
    check_forward(q, k, v, window, sinks, out_dtype=dtype)


BACKWARD = [c for c in FORWARD if c[6] != 256] + [
    (BF, 1, 16, 1, 400, 400, 128, 100, 4),          # one key/value head for all, blocks cut into items
    (BF, 1, 1, 1, 6000, 6000, 64, 50, 4),           # sinks that very many rows see
    (HF, 1, 4, 2, 2000, 2000, 128, 1500, 200),
]


@pytest.mark.parametrize("case", BACKWARD, ids=lambda c: f"{str(c[0])[6:]}-{c[1]}x{c[2]}.{c[3]}x{c[4]}.{c[5]}x{c[6]}-w{c[7]}-s{c[8]}")
@pytest.mark.parametrize("half", [False, True])
def test_backward(case, half):
    dtype, B, H, Hkv, Nq, Nk, d, window, sinks = case
    q, k, v = inputs(dtype, B, H, Hkv, Nq, Nk, d)
    do = normal((B, H, Nq, d), dtype, 4)
    kind = dtype if half else F32
    o, lse = fa2.forward_window(q, k, v, window, sinks, out_dtype=kind)
    grads = fa2.backward_window(q, k, v, o, lse, do, window, sinks, grad_dtype=kind)
    ref, bounds = backward(q, k, v, do, seen(Nq, Nk, window, sinks), 1.0 / math.sqrt(d), EPS[kind] if half else 0.0,
                           EPS[kind])
    for name, g, r, b in zip(("dQ", "dK", "dV"), grads, ref, bounds):
        assert g.dtype is kind
        close(g, r, b, name)
    again = fa2.backward_window(q, k, v, o, lse, do, window, sinks, grad_dtype=kind)
    assert torch.equal(again[1], grads[1]) and torch.equal(again[2], grads[2])
    close(again[0], ref[0], bounds[0], "dQ again")


def test_gradients_against_differences():
    """Central differences of sum(c * O) of the 64-bit form; the gradients carry the kernel's roundings (u each of P,
    dS and O in D), the differences step^2 terms far below them."""
    q, k, v = inputs(HF, 1, 2, 1, 40, 40, 64, std=0.5)
    c = normal(q.shape, HF, 5)
    mask, scale = seen(40, 40, 7, 2), 0.125
    o, lse = fa2.forward_window(q, k, v, 7, 2, scale=scale)
    grads = fa2.backward_window(q, k, v, o, lse, c, 7, 2, scale=scale)
    ref, bounds = backward(q, k, v, c, mask, scale, 0.0, 0.0)
    f = lambda *t: (c.double() * forward_64(*t)).sum().item()  # noqa: E731

    def forward_64(*t):
        kk, vv = (x.double().repeat_interleave(2, 1) for x in t[1:])
        s = (t[0].double() @ kk.transpose(-1, -2) * scale).masked_fill(~mask, -math.inf)
        return torch.softmax(s, -1) @ vv

    tensors = [t.double() for t in (q, k, v)]
    for which in range(3):
        for e in range(0, tensors[which].numel(), 397):
            step = torch.zeros(tensors[which].numel(), dtype=torch.float64, device="cuda")
            step[e] = 1e-4
            step = step.view(tensors[which].shape)
            up = [t + step if i == which else t for i, t in enumerate(tensors)]
            down = [t - step if i == which else t for i, t in enumerate(tensors)]
            slope = (f(*up) - f(*down)) / 2e-4
            assert abs(slope - grads[which].view(-1)[e].item()) <= bounds[which].view(-1)[e].item() + 1e-6


def test_a_window_of_everything_is_causal_attention():
    q, k, v = inputs(BF, 2, 3, 3, 500, 500, 128)
    do = normal(q.shape, BF, 4)
    o, lse = fa2.forward(q, k, v, causal=True)
    # both lie within their bounds of the 64-bit form, but not at the same place: the exponents' offsets differ
    _, _, bO, bL, _, _ = forward(q, k, v, seen(500, 500, 500, 0), 1.0 / math.sqrt(128), EPS[F32])
    for window, sinks in ((500, 0), (1 << 40, 7), (1, 500)):
        ow, lw = fa2.forward_window(q, k, v, window, sinks)
        close(ow, o.double(), 2 * bO)
        close(lw, lse.double(), 2 * bL)
    dk, dv = fa2.backward(q, k, v, o, lse, do, causal=True)[1:]
    got = fa2.backward_window(q, k, v, o, lse, do, 500)
    # the same tiles in the same order, but cut into items and added up in fp32
    _, bounds = backward(q, k, v, do, seen(500, 500, 500, 0), 1.0 / math.sqrt(128), 0.0, 0.0)
    for a, b, bound in zip(got[1:], (dk, dv), bounds[1:]):
        close(a, b.double(), 2.0 ** -10 * bound + 1e-6)


def test_masked_keys_do_not_count_whatever_their_size():
    """Keys outside a row's window that would take all its weight; the largest finite values of the type."""
    big = torch.finfo(HF).max
    q, k, v = inputs(HF, 1, 2, 2, 600, 600, 64)
    for at in (10, 100):                       # (not sinks, far before the last rows)
        k[:, :, at] = big / 64 * q[:, :, 500].sign()
    v[:, :, 100] = big
    window = 200
    o, lse = check_forward(q, k, v, window, 0)
    rows = slice(100 + window, None)           # nobody here sees the large values: weights of exactly 0
    keep = seen(600, 600, window, 0)
    k2, v2 = k.clone(), v.clone()
    k2[:, :, :101], v2[:, :, :101] = 0, 0
    assert torch.equal(fa2.forward_window(q, k2, v2, window)[0][:, :, rows], o[:, :, rows]) and keep.any()


def test_nan_scores_are_not_hidden():
    q, k, v = inputs(BF, 1, 1, 1, 300, 300, 64)
    q[:, :, 7] = float("nan")
    o, lse = fa2.forward_window(q, k, v, 50, 2)
    assert o[0, 0, 7].isnan().all() and lse[0, 0, 7].isnan()
    rest = torch.arange(300, device="cuda") != 7
    assert o[:, :, rest].isfinite().all() and lse[:, :, rest].isfinite().all()


def test_no_rows_and_no_keys():
    for B, H, Hkv, Nq, Nk in ((0, 4, 2, 5, 5), (2, 0, 0, 5, 5), (2, 4, 2, 0, 5), (2, 4, 2, 0, 0)):
        q, k, v = inputs(BF, B, H, Hkv, Nq, Nk, 64)
        o, lse = fa2.forward_window(q, k, v, 3)
        assert o.shape == q.shape and lse.shape == q.shape[:3]
        dk = torch.full(k.shape, 7.0, device="cuda")
        dq, dk, dv = fa2.backward_window(q, k, v, o, lse, q, 3, dk=dk)
        assert dq.shape == q.shape and not dk.any() and not dv.any()
    q, k, v = inputs(BF, 1, 2, 2, 5, 0, 64)
    with pytest.raises(fa2.FA2Error):
        fa2.forward_window(q, k, v, 3)


def test_streams_given_buffers_and_capture():
    q, k, v = inputs(BF, 1, 4, 2, 700, 700, 128)
    do = normal(q.shape, BF, 4)
    o, lse = fa2.forward_window(q, k, v, 100, 4)
    grads = fa2.backward_window(q, k, v, o, lse, do, 100, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    size = fa2.library().fa2_backward_window_workspace_bytes(1, 4, 2, 700, 700, 128, 100, 4, fa2.FA2_DTYPE_FP32)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    g2 = [torch.empty_like(g) for g in grads]
    for handle in (s, s.cuda_stream):
        fa2.forward_window(q, k, v, 100, 4, out=o2, lse=lse2, stream=handle)
        fa2.backward_window(q, k, v, o2, lse2, do, 100, 4, dq=g2[0], dk=g2[1], dv=g2[2], workspace=ws, stream=handle)
        s.synchronize()
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
        assert torch.equal(g2[1], grads[1]) and torch.equal(g2[2], grads[2])
    with pytest.raises(fa2.FA2Error):
        fa2.backward_window(q, k, v, o, lse, do, 100, 4, workspace=ws[:size // 2].clone())
    # captured, and replayed with other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            oc, lc = fa2.forward_window(q, k, v, 100, 4)
            gc = fa2.backward_window(q, k, v, oc, lc, do, 100, 4)
    q.copy_(normal(q.shape, BF, 9))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    o, lse = fa2.forward_window(q, k, v, 100, 4)
    grads = fa2.backward_window(q, k, v, o, lse, do, 100, 4)
    assert torch.equal(oc, o) and torch.equal(lc, lse)
    assert torch.equal(gc[1], grads[1]) and torch.equal(gc[2], grads[2])


def test_a_layer_with_normed_heads():
    """Heads normed and rotated, windowed attention, and the gradients all the way back, as a training step runs them:
    against autograd of the same in 64 bits, each gradient within its roundings (measured against the gradient's
    norm: u for each of the stages' outputs, normed q and k, P, dS, O, dQ, their rotated gradient)."""
    B, H, Hkv, N, d, window, sinks = 1, 4, 2, 300, 64, 90, 3
    x, y, v = normal((B, H, N, d), BF, 1), normal((B, Hkv, N, d), BF, 2), normal((B, Hkv, N, d), BF, 3)
    wq, wk = normal((d,), F32, 5, 0.2) + 1, normal((d,), F32, 6, 0.2) + 1
    do = normal((B, H, N, d), BF, 4)
    pos, freq = torch.arange(N, device="cuda"), fa2.rope_inv_freq(d, device="cuda")
    q, k = fa2.norm_rope(x, wq, pos, freq), fa2.norm_rope(y, wk, pos, freq)
    o, lse = fa2.forward_window(q, k, v, window, sinks, out_dtype=BF)
    dq, dk, dv = fa2.backward_window(q, k, v, o, lse, do, window, sinks, grad_dtype=BF)
    dx, dwq = fa2.norm_rope_backward(dq, x, wq, pos, freq)
    dy, dwk = fa2.norm_rope_backward(dk, y, wk, pos, freq)
    leaves = [t.double().requires_grad_() for t in (x, y, v, wq, wk)]

    def turned(t, w):
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
        a = pos.double()[:, None] * freq[None]
        t0, t1 = t[..., :d // 2], t[..., d // 2:]
        return torch.cat([t0 * a.cos() - t1 * a.sin(), t1 * a.cos() + t0 * a.sin()], -1)

    qq, kk = turned(leaves[0], leaves[3]), turned(leaves[1], leaves[4]).repeat_interleave(2, 1)
    s = (qq @ kk.transpose(-1, -2) / 8.0).masked_fill(~seen(N, N, window, sinks), -math.inf)
    out = torch.softmax(s, -1) @ leaves[2].repeat_interleave(2, 1)
    out.backward(do.double())
    for got, leaf in zip((dx, dy, dv, dwq, dwk), leaves):
        off = (got.double() - leaf.grad).norm() / leaf.grad.norm()
        # ten roundings of at most u each; q's and k's rounding moves a score by up to about 2 u |s|, |s| <= 8
        assert off <= (10 + 2 * 8) * EPS[BF], off

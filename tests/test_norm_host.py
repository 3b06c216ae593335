"""The normed rotary entry points refuse bad arguments on the host, before any GPU work."""
import ctypes

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from exact_attention_17_gb300 import paged
from test_paged_host import BAD_CACHES, cache

BF16, FP16, FP32 = fa2.FA2_DTYPE_BF16, fa2.FA2_DTYPE_FP16, fa2.FA2_DTYPE_FP32


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return fa2.library()


def strides(t, n):
    return None if t is None else (ctypes.c_longlong * n)(*t)


def forward(X=16, xs=(0, 64, 64), Y=4096, ys=(0, 64, 64), B=1, H=1, N=4, d=64, w=16, wt=BF16, eps=1e-6, pos=16, pos64=0,
            ps=0, freq=16, r=64, inter=0, m=1.0, dtype=BF16):
    return fa2.library().fa2_norm_rope(X, strides(xs, 3), Y, strides(ys, 3), B, H, N, d, w, wt, eps, pos, pos64, ps, freq,
                                       r, inter, m, dtype, None)


def backward(G=16, gs=(0, 64, 64), X=16, xs=(0, 64, 64), Y=4096, ys=(0, 64, 64), B=1, H=1, N=4, d=64, w=16, wt=BF16,
             eps=1e-6, pos=16, pos64=0, ps=0, freq=16, r=64, inter=0, m=1.0, dtype=BF16, dw=16, ws=256, size=1 << 20):
    return fa2.library().fa2_norm_rope_backward(G, strides(gs, 3), X, strides(xs, 3), Y, strides(ys, 3), B, H, N, d, w,
                                                wt, eps, pos, pos64, ps, freq, r, inter, m, dtype, dw, ws, size, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_sizes_types_and_pointers(call):
    for bad in (dict(B=-1), dict(H=-1), dict(N=-1), dict(r=66), dict(r=3), dict(r=-2), dict(xs=(0, 64, -64)),
                dict(ys=(0, 64, 0)), dict(ys=(0, 64, 32)), dict(xs=(0, 64, 1 << 40)), dict(B=2, ys=(256, 64, 64), ps=-1),
                dict(B=2, H=4, ys=(64, 64, 256))):
        assert call(**bad) == fa2.FA2_ERR_SHAPE, bad
    for d in (32, 63, 96, 512):
        assert call(d=d, r=2) == fa2.FA2_ERR_HEADDIM
    for bad in (dict(dtype=5), dict(wt=FP16), dict(wt=9), dict(dtype=FP32)):
        assert call(**bad) == fa2.FA2_ERR_DTYPE, bad
    for bad in (dict(m=float("inf")), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call(**bad) == fa2.FA2_ERR_SCALE, bad
    for bad in (dict(X=None), dict(Y=None), dict(pos=None), dict(freq=None), dict(w=None), dict(xs=None), dict(ys=None)):
        assert call(**bad) == fa2.FA2_ERR_NULL, bad
    for bad in (dict(X=17), dict(Y=4097), dict(pos=2), dict(pos=4, pos64=1), dict(freq=4), dict(w=17),
                dict(w=18, wt=FP32)):
        assert call(**bad) == fa2.FA2_ERR_ALIGN, bad


def test_the_gradients_own_arguments():
    for bad in (dict(G=None), dict(gs=None), dict(dw=None), dict(ws=None)):
        assert backward(**bad) == fa2.FA2_ERR_NULL, bad
    for bad in (dict(G=17), dict(dw=2), dict(ws=128)):
        assert backward(**bad) == fa2.FA2_ERR_ALIGN, bad
    assert backward(gs=(0, -64, 64), H=2) == fa2.FA2_ERR_SHAPE
    assert fa2.library().fa2_norm_rope_backward_workspace_bytes(96) == 0


def test_empty_calls():
    for empty in (dict(B=0), dict(H=0), dict(N=0, X=None)):
        assert forward(**empty) == fa2.FA2_OK


def append(c, K=16, ks=(128, 64), V=16, vs=(128, 64), Q=16, qs=(256, 64), Qo=4096, qos=(256, 64), Hq=4, cu=None, T=2,
           qw=16, kw=16, wt=BF16, eps=1e-6, freq=16, r=64, m=1.0):
    return fa2.library().fa2_append_paged_norm(None if c is None else ctypes.byref(c), K, strides(ks, 2), V,
                                               strides(vs, 2), Q, strides(qs, 2), Qo, strides(qos, 2), Hq, cu, T, qw, kw,
                                               wt, eps, freq, r, 0, m, None)


def test_append():
    for bad, code in BAD_CACHES:
        if "dtype" not in bad:
            assert append(cache(**bad)) == getattr(fa2, "FA2_ERR_" + code), bad
    c = cache()
    for bad in (dict(wt=FP16), dict(wt=7)):
        assert append(c, **bad) == fa2.FA2_ERR_DTYPE, bad
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(m=float("nan"))):
        assert append(c, **bad) == fa2.FA2_ERR_SCALE, bad
    for bad in (dict(qw=17), dict(kw=17), dict(qw=18, wt=FP32), dict(kw=18, wt=FP32), dict(K=8), dict(cu=2)):
        assert append(c, **bad) == fa2.FA2_ERR_ALIGN, bad
    for bad in (dict(T=-1), dict(T=3), dict(r=66), dict(ks=(32, 64))):
        assert append(c, **bad) == fa2.FA2_ERR_SHAPE, bad
    for bad in (dict(K=None), dict(Q=None), dict(freq=None)):
        assert append(c, **bad) == fa2.FA2_ERR_NULL, bad
    assert append(c, T=0, K=None) == fa2.FA2_OK


@pytest.fixture(params=["binding", "ctypes"])
def way(request, monkeypatch):
    if paged.torch is None:
        paged._load()
    if request.param == "ctypes":
        monkeypatch.setattr(paged, "_fast", None)


def test_python_calls_check_their_tensors(way):
    x, w = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(64)
    pos, freq = torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    for call in (lambda: fa2.norm_rope(x, w, pos, freq), lambda: fa2.norm_rope_backward(x, x, w, pos, freq)):
        with pytest.raises(ValueError, match="CUDA"):
            call()

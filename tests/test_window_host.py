"""The window entry points refuse bad arguments on the host, before any GPU work."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild

BF16, FP16, FP32 = fa2.FA2_DTYPE_BF16, fa2.FA2_DTYPE_FP16, fa2.FA2_DTYPE_FP32


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return fa2.library()


def forward(Q=16, K=16, V=16, O=16, L=16, B=1, H=4, Hkv=2, Nq=8, Nk=8, d=64, window=4, sinks=0, scale=0.125, t=BF16,
            ot=FP32):
    return fa2.library().fa2_forward_window(Q, K, V, O, L, B, H, Hkv, Nq, Nk, d, window, sinks, scale, t, ot, None)


def backward(Q=16, K=16, V=16, O=16, G=16, L=16, dQ=16, dK=16, dV=16, B=1, H=4, Hkv=2, Nq=8, Nk=8, d=64, window=4,
             sinks=0, scale=0.125, t=BF16, ot=FP32, gt=FP32, ws=256, size=1 << 20):
    return fa2.library().fa2_backward_window(Q, K, V, O, G, L, dQ, dK, dV, B, H, Hkv, Nq, Nk, d, window, sinks, scale, t,
                                             ot, gt, ws, size, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_common_refusals(call):
    for bad in (dict(B=-1), dict(H=-4), dict(Hkv=-1), dict(Nq=-1), dict(Nk=-1), dict(Nk=0), dict(window=0),
                dict(window=-3), dict(sinks=-1), dict(Hkv=0), dict(H=3), dict(H=0), dict(B=1 << 30)):
        assert call(**bad) == fa2.FA2_ERR_SHAPE, bad
    for bad in (dict(t=FP32), dict(t=7), dict(ot=FP16), dict(ot=5)):
        assert call(**bad) == fa2.FA2_ERR_DTYPE, bad
    assert call(d=96) == fa2.FA2_ERR_HEADDIM
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=s) == fa2.FA2_ERR_SCALE
    for name in ("Q", "K", "V", "O", "L"):
        assert call(**{name: None}) == fa2.FA2_ERR_NULL, name
        assert call(**{name: 18}) == fa2.FA2_ERR_ALIGN, name
    for empty in (dict(B=0), dict(H=0, Hkv=0), dict(Nq=0, Nk=0)):
        assert call(**empty) == fa2.FA2_OK, empty


def test_the_gradients_own_refusals():
    assert backward(d=256) == fa2.FA2_ERR_HEADDIM
    for bad in (dict(gt=FP16), dict(gt=9)):
        assert backward(**bad) == fa2.FA2_ERR_DTYPE
    for name in ("G", "dQ", "dK", "dV", "ws"):
        assert backward(**{name: None}) == fa2.FA2_ERR_NULL, name
    for name, at in (("G", 8), ("dQ", 8), ("dK", 8), ("dV", 8), ("ws", 128)):
        assert backward(**{name: at}) == fa2.FA2_ERR_ALIGN, name
    f = fa2.library().fa2_backward_window_workspace_bytes
    for bad in ((1, 4, 2, 8, 8, 96, 4, 0, FP32), (1, 4, 3, 8, 8, 64, 4, 0, FP32), (1, 4, 2, 8, 8, 64, 0, 0, FP32),
                (1, 4, 2, 0, 8, 64, 4, 0, FP32)):
        assert f(*bad) == 0


def test_python_calls_check_their_tensors():
    q, k = torch.zeros(1, 4, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa2.forward_window(q, k, k, 4)
    with pytest.raises(ValueError, match="CUDA"):
        fa2.backward_window(q, k, k, q, q, q, 4)

"""Normed heads with an eps of zero, and rows that leave a block's tokens unfilled."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import release_memory
from test_norm_gpu import BF, F32, HF, backward_64, close, forward_64, normal, rounded

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


# 1e-60 is zero in fp32.  Rotary 16 columns fill whole 16-byte vectors of every type and layout, 20 none but
# interleaved fp32's.  A block has 8 to 64 tokens: one token, one less and one more than a block's, and whole blocks.
@pytest.mark.parametrize("eps", [0.0, 1e-60])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [16, 20])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_eps_of_zero(dtype, d, rotary, interleaved, eps):
    freq, w = fa2.rope_inv_freq(rotary, device="cuda"), normal((d,), dtype, 2, std=0.3, mean=1.0)
    for B, H, N in ((1, 1, 1), (1, 3, 7), (3, 2, 21), (1, 2, 65), (2, 2, 64)):
        x, dy = normal((B, H, N, d), dtype, seed=N), normal((B, H, N, d), dtype, seed=3)
        pos = torch.arange(N, device="cuda")
        how = dict(eps=eps, interleaved=interleaved, mscale=1.0)
        y = fa2.norm_rope(x, w, pos, freq, **how)
        ref, bound, size = forward_64(x, w, pos, freq, **how)
        close(y, ref, rounded(bound, size, dtype))
        dx, dw = fa2.norm_rope_backward(dy, x, w, pos, freq, **how)
        # a lane sees the heads of its tokens (a block's places one after the other), then trees and 32 strips
        ref, bound, ref_w, bound_w = backward_64(dy, x, w, pos, freq, **how, chain=H * B * N + 128)
        assert dx.isfinite().all() and dw.isfinite().all(), (B, H, N)
        close(dx, ref, rounded(bound, ref, dtype))
        close(dw, ref_w, bound_w)

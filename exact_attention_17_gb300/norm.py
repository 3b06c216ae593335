"""Each head's row normed and rotated in one pass, and the gradients.

The norm that queries and keys take before their rotary positions: a row x of d
columns (64, 128 or 256) with weight w at position t becomes R(t) (w x r), r =
1 / sqrt(mean(x^2) + eps).  ``append_paged`` does the same on the way into a
paged cache.  This module only marshals arguments, as ``paged`` does.
"""
from __future__ import annotations

from . import paged
from .paged import _answer, _Call, _fail, _heads, _inv_freq_args, _like, _position_args, _weight_args, _workspace_size


def norm_rope(x, weight, positions, inv_freq, eps: float = 1e-6, interleaved: bool = False, mscale: float = 1.0,
              out=None, stream=None):
    """Norm of each head's row, then rotary positions (fa2_norm_rope).

    x [B, H, N, d] with positions [N] or [B, N], or packed x [T, H, d] with
    positions [T] (int32 or int64); bf16, fp16 or fp32.  ``weight`` [d] is of x's
    type or fp32.  ``inv_freq``, ``interleaved`` and ``mscale`` as ``rope`` (None
    for ``inv_freq``: no rotation).  ``out=x`` works in place.
    """
    if paged.torch is None:
        paged._load()
    if paged._fast is not None and out is None and stream is None:
        r = paged._fast.norm_rope(x, weight, positions, inv_freq, eps, interleaved, mscale)
        if r is not None:
            return _answer(r, "fa2_norm_rope")
    B, H, N, d, xs = _heads("x", x)
    device = x.device
    place = _position_args(positions, B, N, x.dim(), device)
    w, code = _weight_args("weight", weight, d, x.dtype, device)
    freq, rotary_dim = _inv_freq_args(inv_freq, device, d)
    with _Call(device, stream) as handle:
        if out is None:
            out = paged.torch.empty(x.shape, dtype=x.dtype, device=device)
        rc = paged._lib.fa2_norm_rope(x.data_ptr(), xs, out.data_ptr(), _like("out", out, x), B, H, N, d, w, code, eps,
                                      *place, freq, rotary_dim, 1 if interleaved else 0, mscale,
                                      paged._codes[x.dtype], handle)
    if rc:
        _fail(rc, "fa2_norm_rope")
    return out


def norm_rope_backward(dy, x, weight, positions, inv_freq, eps: float = 1e-6, interleaved: bool = False,
                       mscale: float = 1.0, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of ``norm_rope`` for the upstream gradient ``dy`` (fa2_norm_rope_backward).

    dy as x; the other arguments are those of the forward call.  Returns (dx of
    x's type, dweight fp32 [d], the sum over all rows).  ``dx=dy`` and ``dx=x``
    work in place.  The workspace (a uint8 CUDA tensor) is allocated here unless
    given; calls that may overlap need one each.
    """
    if paged.torch is None:
        paged._load()
    if paged._fast is not None and dx is None and dweight is None and workspace is None and stream is None:
        r = paged._fast.norm_rope_backward(dy, x, weight, positions, inv_freq, eps, interleaved, mscale)
        if r is not None:
            return _answer(r, "fa2_norm_rope_backward")
    torch = paged.torch
    B, H, N, d, xs = _heads("x", x)
    device = x.device
    gs = _like("dy", dy, x)
    place = _position_args(positions, B, N, x.dim(), device)
    w, code = _weight_args("weight", weight, d, x.dtype, device)
    freq, rotary_dim = _inv_freq_args(inv_freq, device, d)
    with _Call(device, stream) as handle:
        if dx is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=device)
        ys = _like("dx", dx, x)
        if dweight is None:
            dweight = torch.empty(d, dtype=torch.float32, device=device)
        elif (dweight.dtype is not torch.float32 or dweight.shape != (d,) or not dweight.is_contiguous()
              or dweight.device != device):
            raise ValueError(f"dweight must be a contiguous fp32 tensor of shape {(d,)} on {device}")
        if workspace is None:
            with torch.cuda.device(device):
                size = paged._lib.fa2_norm_rope_backward_workspace_bytes(d)
            workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
        else:
            size = _workspace_size(workspace, device)
        rc = paged._lib.fa2_norm_rope_backward(dy.data_ptr(), gs, x.data_ptr(), xs, dx.data_ptr(), ys, B, H, N, d, w,
                                               code, eps, *place, freq, rotary_dim, 1 if interleaved else 0, mscale,
                                               paged._codes[x.dtype], dweight.data_ptr(), workspace.data_ptr(), size,
                                               handle)
    if rc:
        _fail(rc, "fa2_norm_rope_backward")
    return dx, dweight

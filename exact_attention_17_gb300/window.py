"""Causal attention of which each query sees its last keys and the first few.

Query i sees the keys j <= i with i - j < window (its own among them) or j <
sinks.  Query heads share key/value heads in groups.  ``forward_paged_window`` is
the same over a paged cache.  This module only marshals arguments, as ``paged``
does.
"""
from __future__ import annotations

from . import paged
from .paged import _answer, _Call, _default_scale, _fail, _sizes, _workspace_size


def _dense(name, t, shape, dtype, device):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _output(name, t, shape, dtype, device):
    return paged.torch.empty(shape, dtype=dtype, device=device) if t is None else _dense(name, t, shape, dtype, device)


def _reach(window, sinks):
    """As C ints: a window or sinks beyond every length are all of them."""
    window, sinks = min(int(window), (1 << 31) - 1), min(int(sinks), (1 << 31) - 1)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1, sinks not negative")
    return window, sinks


def _arguments(q, k, v, window, sinks, scale):
    """Device, sizes (B, H, Hkv, Nq, Nk, d, window, sinks), scale and type code."""
    torch = paged.torch
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
        raise ValueError("q must be bf16 or fp16")
    if not q.is_cuda or q.dim() != 4 or k.dim() != 4:
        raise ValueError("q [B, H, Nq, d] and k [B, Hkv, Nk, d] must be 4-D CUDA tensors")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    _dense("q", q, q.shape, q.dtype, q.device)
    for name, t in (("k", k), ("v", v)):
        _dense(name, t, (B, Hkv, Nk, d), q.dtype, q.device)
    if (H % Hkv if Hkv else H) != 0:
        raise ValueError(f"{H} query heads are no multiple of {Hkv} key/value heads")
    _sizes(B, H, Hkv, Nq, Nk, d)
    return (B, H, Hkv, Nq, Nk, d, window, sinks), _default_scale(d) if scale is None else scale


def forward_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, out=None, lse=None,
                   out_dtype=None, stream=None):
    """Attention with a window (fa2_forward_window).

    q [B, H, Nq, d]; k, v [B, Hkv, Nk, d] (H a multiple of Hkv: query head h reads
    head h // (H // Hkv)), all bf16 or all fp16, contiguous, on one device; d = 64,
    128 or 256.  Returns (O [B, H, Nq, d], LSE fp32 [B, H, Nq]); O is fp32 unless
    ``out_dtype`` is q's type.  Rows without keys give O = 0 and LSE = -inf.
    ``scale`` defaults to 1/sqrt(d) in float32.
    """
    if paged.torch is None:
        paged._load()
    window, sinks = _reach(window, sinks)
    if paged._fast is not None and out is None and lse is None and stream is None:
        half = out_dtype is not None and out_dtype is not paged.torch.float32
        if not half or out_dtype is q.dtype:
            r = paged._fast.forward_window(q, k, v, window, sinks, scale, half)
            if r is not None:
                return _answer(r, "fa2_forward_window")
    sizes, scale = _arguments(q, k, v, window, sinks, scale)
    torch, device = paged.torch, q.device
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    if out_dtype is not torch.float32 and out_dtype is not q.dtype:
        raise ValueError("out_dtype must be fp32 or q's type")
    with _Call(device, stream) as handle:
        out = _output("out", out, q.shape, out_dtype, device)
        lse = _output("lse", lse, q.shape[:3], torch.float32, device)
        rc = paged._lib.fa2_forward_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                           *sizes, scale, paged._codes[q.dtype], paged._codes[out_dtype], handle)
    if rc:
        _fail(rc, "fa2_forward_window")
    return out, lse


def backward_window(q, k, v, o, lse, do, window: int, sinks: int = 0, scale: float | None = None, dq=None, dk=None,
                    dv=None, grad_dtype=None, workspace=None, stream=None):
    """Gradients of ``forward_window`` (fa2_backward_window).

    ``o`` (fp32 or q's type) and ``lse`` are what the forward pass returned for
    the same arguments, ``do`` [B, H, Nq, d] of q's type.  Returns (dQ, dK, dV) in
    fp32, or in q's type when ``grad_dtype`` says so; dK and dV are summed over the
    query heads that share them.  d = 64 or 128.  The workspace (a uint8 CUDA
    tensor) is allocated here unless given; calls that may overlap need one each.
    """
    if paged.torch is None:
        paged._load()
    window, sinks = _reach(window, sinks)
    if paged._fast is not None and dq is None and dk is None and dv is None and workspace is None and stream is None:
        half = grad_dtype is not None and grad_dtype is not paged.torch.float32
        if not half or grad_dtype is q.dtype:
            r = paged._fast.backward_window(q, k, v, o, lse, do, window, sinks, scale, half)
            if r is not None:
                return _answer(r, "fa2_backward_window")
    sizes, scale = _arguments(q, k, v, window, sinks, scale)
    torch, device = paged.torch, q.device
    grad_dtype = torch.float32 if grad_dtype is None else grad_dtype
    if grad_dtype is not torch.float32 and grad_dtype is not q.dtype:
        raise ValueError("grad_dtype must be fp32 or q's type")
    if o.dtype is not torch.float32:
        _dense("o", o, q.shape, q.dtype, device)
    _dense("o", o, q.shape, o.dtype, device)
    _dense("lse", lse, q.shape[:3], torch.float32, device)
    _dense("do", do, q.shape, q.dtype, device)
    codes = (paged._codes[q.dtype], paged._codes[o.dtype], paged._codes[grad_dtype])
    with _Call(device, stream) as handle:
        dq = _output("dq", dq, q.shape, grad_dtype, device)
        dk = _output("dk", dk, k.shape, grad_dtype, device)
        dv = _output("dv", dv, k.shape, grad_dtype, device)
        if workspace is None:
            with torch.cuda.device(device):
                size = paged._lib.fa2_backward_window_workspace_bytes(*sizes, codes[2])
            workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
        else:
            size = _workspace_size(workspace, device)
        rc = paged._lib.fa2_backward_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
                                            lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *sizes, scale,
                                            *codes, workspace.data_ptr(), size, handle)
    if rc:
        _fail(rc, "fa2_backward_window")
    return dq, dk, dv

"""Attention over a paged key/value cache, and what keeps such a cache.

A cache is a pair of tensors ``k_pages``, ``v_pages`` [P, Hkv, S, d] (P pages of
S slots; any strides with a dense last dimension, so a [P, S, Hkv, d] tensor
passes as ``t.transpose(1, 2)`` and one layer of a larger pool as a view), a
``page_table`` int32 [B, M] and lengths int32 [B].  Sequence b's token t lies in
slot t % S of page ``page_table[b, t // S]``.  New tokens are packed [T, H, d];
``cu_q`` int32 [B + 1] says where each sequence's begin (None: one token for
each sequence).  Lengths count the new tokens too.

Tables, lengths and offsets stay on the device: nothing here waits for the GPU,
and a captured call can be replayed after they changed.  What they hold is
checked where it is used: nothing outside the cache is read or written, and
``fa2_device_status`` reports ``FA2_ERR_PAGE``.

A step of a server, layer by layer::

    missing = fa2.pages_reserve(page_table, lens, refs, new_tokens, S)     # once a step
    q = fa2.append_paged(k, v, k_pages, v_pages, page_table, lens, cu_q=cu_q, q=q, inv_freq=inv_freq)
    o, lse = fa2.forward_paged(q, k_pages, v_pages, page_table, lens, cu_q=cu_q)

This module only marshals arguments (see the package docstring).  Outputs and
workspaces that a call makes belong to the stream that it runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import exact_attention_17_gb300 as fa2

_NULL_CONTEXT = contextlib.nullcontext()


def _on_stream(stream, device):
    """(raw handle, context in which tensors are allocated on that stream)."""
    import torch

    current = torch.cuda.current_stream(device)
    if stream is None:
        return current.cuda_stream, _NULL_CONTEXT
    handle = getattr(stream, "cuda_stream", stream)
    if handle == current.cuda_stream:
        return handle, _NULL_CONTEXT
    if handle == 0:
        return handle, torch.cuda.stream(torch.cuda.default_stream(device))
    return handle, torch.cuda.stream(torch.cuda.ExternalStream(handle, device=device))


def _ints(name, t, shape, device):
    """An int32 CUDA tensor of `shape`, rows dense."""
    import torch

    if (t.dtype is not torch.int32 or tuple(t.shape) != shape or t.device != device
            or (shape and shape[-1] > 1 and t.stride(-1) != 1)):
        raise ValueError(f"{name} must be a dense int32 tensor of shape {shape} on {device}")


def _rows(name, t, shape, dtype, device):
    """A [T, H, d] tensor of the cache's type, last dimension dense."""
    if t.dtype is not dtype or tuple(t.shape) != shape or t.device != device or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {shape} on {device} with a dense last dimension")


def _cache_args(k_pages, v_pages, page_table, kv_lens):
    import torch

    dtype, device = k_pages.dtype, k_pages.device
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("k_pages must be bf16 or fp16")
    if not k_pages.is_cuda or k_pages.dim() != 4 or k_pages.stride(3) != 1:
        raise ValueError("k_pages must be a 4-D CUDA tensor with a dense last dimension")
    if (v_pages.dtype is not dtype or v_pages.shape != k_pages.shape or v_pages.stride() != k_pages.stride()
            or v_pages.device != device):
        raise ValueError("v_pages must match k_pages in type, shape, strides and device")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, M]")
    B, M = page_table.shape
    _ints("page_table", page_table, (B, M), device)
    _ints("kv_lens", kv_lens, (B,), device)
    P, Hkv, S, d = k_pages.shape
    ps, hs, ss, _ = k_pages.stride()
    return fa2.PagedCacheArgs(k_pages.data_ptr(), v_pages.data_ptr(), P, Hkv, S, d, ps, hs, ss,
                              fa2._dtype_codes()[dtype], page_table.data_ptr(), page_table.stride(0), M, B,
                              kv_lens.data_ptr())


def _check_offsets(cu_q, B, T, device):
    if cu_q is not None:
        _ints("cu_q", cu_q, (B + 1,), device)
    elif T != B:
        raise ValueError(f"without cu_q there is one new token for each of the {B} sequences, not {T}")


def forward_paged(q, k_pages, v_pages, page_table, kv_lens, cu_q=None, causal: bool = True,
                  scale: float | None = None, out=None, lse=None, out_dtype=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache (fa2_forward_paged).

    q [T, Hq, d] of the cache's type (Hq a multiple of Hkv: query head h reads
    key/value head h // (Hq // Hkv)); token i of sequence b sits at position
    kv_lens[b] - c_b + i and, when causal, sees the keys up to its own.
    Returns (O [T, Hq, d], LSE fp32 [T, Hq]); O in q's type, or fp32 with
    ``out_dtype``.  Rows without keys give O = 0 and LSE = -inf; rows behind
    cu_q[B] are not written.  ``scale`` defaults to 1/sqrt(d) in float32.  The
    workspace (a uint8 CUDA tensor) is allocated here unless given; calls that
    may overlap need one each.
    """
    import torch

    args = _cache_args(k_pages, v_pages, page_table, kv_lens)
    dtype, device = k_pages.dtype, k_pages.device
    if q.dim() != 3 or q.shape[2] != args.d:
        raise ValueError(f"q must be [T, Hq, {args.d}]")
    T, Hq, d = q.shape
    _rows("q", q, (T, Hq, d), dtype, device)
    if Hq % args.kv_heads != 0:
        raise ValueError(f"{Hq} query heads are no multiple of {args.kv_heads} key/value heads")
    _check_offsets(cu_q, args.B, T, device)
    out_dtype = dtype if out_dtype is None else out_dtype
    if out_dtype is not torch.float32 and out_dtype is not dtype:
        raise ValueError("out_dtype must be fp32 or the cache's type")
    if scale is None:
        scale = _default_scale(d)
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        need = fa2.library().fa2_forward_paged_workspace_bytes(args.B, T, Hq, args.kv_heads, d, cu_q is not None)
        with here:
            if out is None:
                out = torch.empty((T, Hq, d), dtype=out_dtype, device=device)
            if lse is None:
                lse = torch.empty((T, Hq), dtype=torch.float32, device=device)
            if workspace is None:
                workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
        if out.dtype is not out_dtype or out.shape != (T, Hq, d) or not out.is_contiguous() or out.device != device:
            raise ValueError(f"out must be a contiguous {out_dtype} tensor of shape {(T, Hq, d)} on {device}")
        if (lse.dtype is not torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()
                or lse.device != device):
            raise ValueError(f"lse must be a contiguous fp32 tensor of shape {(T, Hq)} on {device}")
        if not workspace.is_contiguous() or workspace.device != device:
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        rc = fa2.library().fa2_forward_paged(
            ctypes.byref(args), q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), lse.data_ptr(),
            None if cu_q is None else cu_q.data_ptr(), T, Hq, int(bool(causal)), float(scale),
            fa2._dtype_codes()[out_dtype], workspace.data_ptr(), workspace.numel() * workspace.element_size(), handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_forward_paged")
    return out, lse


_scales = {}


def _default_scale(d):
    """1/sqrt(d) rounded once to float32."""
    if d not in _scales:
        _scales[d] = ctypes.c_float(1.0 / math.sqrt(d)).value
    return _scales[d]


def _inv_freq_args(inv_freq, device, d):
    import torch

    if inv_freq is None:
        return None, 0
    if (inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous()
            or inv_freq.device != device):
        raise ValueError(f"inv_freq must be a contiguous 1-D float64 tensor on {device}")
    if 2 * inv_freq.numel() > d:
        raise ValueError(f"inv_freq holds more than the {d // 2} pairs of a head")
    return inv_freq.data_ptr(), 2 * inv_freq.numel()


def _strides(t):
    return (ctypes.c_longlong * 2)(t.stride(0), t.stride(1))


def append_paged(k, v, k_pages, v_pages, page_table, kv_lens, cu_q=None, q=None, q_out=None, inv_freq=None,
                 interleaved: bool = False, mscale: float = 1.0, stream=None):
    """Write new tokens into a paged cache (fa2_append_paged).

    k, v [T, Hkv, d] go to their sequences' pages at positions kv_lens[b] - c_b
    + i (the pages must be there: ``pages_reserve``), k rotated at its position
    when ``inv_freq`` is given (see ``rope``).  With ``q`` [T, Hq, d] the
    queries are rotated in the same launch and returned (``q_out``; pass
    ``q_out=q`` to rotate in place).  Rows behind cu_q[B] are not touched.
    """
    import torch

    args = _cache_args(k_pages, v_pages, page_table, kv_lens)
    dtype, device = k_pages.dtype, k_pages.device
    if k.dim() != 3:
        raise ValueError(f"k must be [T, {args.kv_heads}, {args.d}]")
    T, shape = k.shape[0], (k.shape[0], args.kv_heads, args.d)
    _rows("k", k, shape, dtype, device)
    _rows("v", v, shape, dtype, device)
    _check_offsets(cu_q, args.B, T, device)
    Hq = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be [{T}, Hq, {args.d}]")
        Hq = q.shape[1]
        _rows("q", q, (T, Hq, args.d), dtype, device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    freq, rotary_dim = _inv_freq_args(inv_freq, device, args.d)
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        if q is not None and q_out is None:
            with here:
                q_out = torch.empty((T, Hq, args.d), dtype=dtype, device=device)
        if q is not None:
            _rows("q_out", q_out, (T, Hq, args.d), dtype, device)
        rc = fa2.library().fa2_append_paged(
            ctypes.byref(args), k.data_ptr(), _strides(k), v.data_ptr(), _strides(v),
            None if q is None else q.data_ptr(), None if q is None else _strides(q),
            None if q is None else q_out.data_ptr(), None if q is None else _strides(q_out), Hq,
            None if cu_q is None else cu_q.data_ptr(), T, freq, rotary_dim, int(bool(interleaved)), float(mscale),
            handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_append_paged")
    return q_out


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                  original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Radians per position of each rotated pair, float64 [rotary_dim // 2].

    base ** (-2 i / rotary_dim), scaled for contexts ``factor`` times the trained
    ``original_length``:

    * ``"linear"``: every frequency divided by the factor;
    * ``"base"``: the base times factor ** (r / (r - 2)), which divides the
      slowest pair's frequency by the factor and leaves the fastest one;
    * ``"ramp"``: pairs that turn at least ``beta_fast`` times within
      original_length stay, those that turn less than ``beta_slow`` times are
      divided by the factor, linear in the pair's number between; usually with
      ``mscale = 0.1 ln(factor) + 1``.
    """
    import torch

    r = rotary_dim
    if r < 2 or r % 2 != 0:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (base > 1.0 and factor >= 1.0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "base":
        if r < 4:
            raise ValueError("scaling the base needs at least two pairs")
        base = base * factor ** (r / (r - 2))
    freq = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "ramp":
        def pair(turns):   # the pair that turns so often within original_length
            return r * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        low = max(math.floor(pair(beta_fast)), 0)
        high = min(math.ceil(pair(beta_slow)), r - 1)
        weight = [min(1.0, max(0.0, (i - low) / max(high - low, 0.001))) for i in range(r // 2)]
        freq = [f * (1 - w) + f / factor * w for f, w in zip(freq, weight)]
    return torch.tensor(freq, dtype=torch.float64, device=device)


def _rope(x, positions, inv_freq, interleaved, mscale, out, stream, transposed):
    import torch

    codes = fa2._dtype_codes()
    if x.dtype not in codes or not x.is_cuda or x.dim() not in (3, 4) or x.stride(-1) != 1:
        raise ValueError("x must be a bf16, fp16 or fp32 CUDA tensor [T, H, d] or [B, H, N, d], last dimension dense")
    device = x.device
    if x.dim() == 3:     # [T, H, d]: one batch, tokens outside the heads
        B, N, H, d = 1, *x.shape
    else:
        B, H, N, d = x.shape
    if positions.dtype not in (torch.int32, torch.int64) or positions.device != device:
        raise ValueError(f"positions must be int32 or int64 on {device}")
    if tuple(positions.shape) not in ((N,), (B, N)) or (N > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions must be a dense [{N}]" + (f" or [{B}, {N}]" if x.dim() == 4 else ""))
    freq, rotary_dim = _inv_freq_args(inv_freq, device, d)
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        if out is None:
            with here:
                out = torch.empty(x.shape, dtype=x.dtype, device=device)
        if out.dtype is not x.dtype or out.shape != x.shape or out.device != device or out.stride(-1) != 1:
            raise ValueError(f"out must be a {x.dtype} tensor of shape {tuple(x.shape)} on {device}, last dimension dense")

        def strides(t):   # {batch, head, token}
            s = (0, t.stride(1), t.stride(0)) if t.dim() == 3 else t.stride()[:3]
            return (ctypes.c_longlong * 3)(*s)

        rc = fa2.library().fa2_rope(
            x.data_ptr(), strides(x), out.data_ptr(), strides(out), B, H, N, d, positions.data_ptr(),
            int(positions.dtype is torch.int64), positions.stride(0) if positions.dim() == 2 else 0, freq, rotary_dim,
            int(bool(interleaved)), float(mscale), int(transposed), codes[x.dtype], handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_rope")
    return out


def rope(x, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, out=None, stream=None):
    """Rotary positions (fa2_rope).

    x [B, H, N, d] with positions [N] or [B, N], or packed x [T, H, d] with
    positions [T] (int32 or int64); bf16, fp16 or fp32.  The first 2 *
    len(inv_freq) columns are rotated: columns (i, i + len(inv_freq)), or (2i,
    2i + 1) when ``interleaved``, by position * inv_freq[i] radians
    (``rope_inv_freq``), times ``mscale``; the others are copied.  ``out=x``
    works in place.
    """
    return _rope(x, positions, inv_freq, interleaved, mscale, out, stream, False)


def rope_backward(do, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, out=None, stream=None):
    """Gradient of ``rope`` with respect to x for the upstream gradient ``do``
    (the transposed rotation); arguments as ``rope``."""
    return _rope(do, positions, inv_freq, interleaved, mscale, out, stream, True)


def _tables(page_table, lens, refs, page_size):
    device = page_table.device
    if page_table.dim() != 2 or not page_table.is_cuda or refs.dim() != 1:
        raise ValueError("page_table must be a CUDA tensor [B, M], refs [P]")
    B, M = page_table.shape
    _ints("page_table", page_table, (B, M), device)
    _ints("lens", lens, (B,), device)
    _ints("refs", refs, (refs.shape[0],), device)
    return fa2.PageTablesArgs(page_table.data_ptr(), page_table.stride(0), M, B, lens.data_ptr(), refs.data_ptr(),
                              refs.shape[0], page_size), device


def _pools(pools):
    """Page data as an array of planes: a tensor [..., P, Hkv, S, d], or a list of such tensors."""
    import torch

    tensors = [pools] if torch.is_tensor(pools) else list(pools)
    pointers, shape, stride, device = [], None, None, None
    for t in tensors:
        if not t.is_cuda or t.dim() < 4:
            raise ValueError("pools must be CUDA tensors [..., P, Hkv, S, d]")
        page = sorted((st, n) for st, n in zip(t.stride()[-3:], t.shape[-3:]) if n > 1)
        dense = 1
        for st, n in page:
            if st != dense:
                raise ValueError("the elements of a page must be dense")
            dense *= n
        this = (tuple(t.shape[-4:]), t.stride()[-4:], t.dtype, t.device)
        if shape is None:
            shape, stride, device = this, t.stride(-4) * t.element_size(), t.device
        if this != shape:
            raise ValueError("all pools must have the same pages, strides, type and device")
        planes = [t] if t.dim() == 4 else t.flatten(0, -5).unbind(0) if t.dim() == 5 else [
            p for p in _leading(t)]
        pointers += [p.data_ptr() for p in planes]
    if shape is None:
        raise ValueError("pools must hold at least one tensor")
    (P, Hkv, S, d), size = shape[0], tensors[0].element_size()
    array = (ctypes.c_void_p * max(len(pointers), 1))(*pointers)
    args = fa2.PagePoolsArgs(ctypes.cast(array, ctypes.c_void_p), len(pointers), P, stride, Hkv * S * d * size)
    return args, array, S, device


def _leading(t):
    """The [P, Hkv, S, d] planes of a tensor with more leading dimensions."""
    if t.dim() == 4:
        yield t
    else:
        for part in t.unbind(0):
            yield from _leading(part)


def _workspace(num_pages, n, given, device):
    import torch

    need = fa2.library().fa2_pages_workspace_bytes(num_pages, n)
    if given is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    if not given.is_contiguous() or given.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return given


def _size(workspace):
    return workspace.numel() * workspace.element_size()


def pages_reserve(page_table, lens, refs, add, page_size: int, workspace=None, stream=None):
    """Make room for ``add`` int32 [B] more tokens (fa2_pages_reserve).

    ``lens`` grows by ``add`` and ``page_table`` by the pages that takes, the
    free ones (``refs`` [P] == 0) of the lowest numbers.  Returns an int32 CUDA
    tensor [1]: 0, or the number of pages that lack, or -1 where a table row is
    too short -- then nothing has changed.
    """
    import torch

    args, device = _tables(page_table, lens, refs, page_size)
    _ints("add", add, (args.B,), device)
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        with here:
            workspace = _workspace(args.num_pages, 0, workspace, device)
            missing = torch.empty(1, dtype=torch.int32, device=device)
        rc = fa2.library().fa2_pages_reserve(ctypes.byref(args), add.data_ptr(), missing.data_ptr(),
                                             workspace.data_ptr(), _size(workspace), handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_pages_reserve")
    return missing


def _pair_lists(src, dst, device):
    n = src.shape[0] if src.dim() == 1 else -1
    _ints("src", src, (n,), device)
    _ints("dst", dst, (n,), device)
    return n


def pages_fork(page_table, lens, refs, src, dst, pools, workspace=None, stream=None):
    """Sequences ``dst`` (empty) become copies of ``src``, int32 [n] (fa2_pages_fork).

    Full pages are shared, a partly filled last page is copied in every plane of
    ``pools`` (a tensor [..., P, Hkv, S, d] or a list of them: all the layers' K
    and V).  Returns the pages that lack as ``pages_reserve`` does.
    """
    import torch

    data, array, S, pool_device = _pools(pools)
    args, device = _tables(page_table, lens, refs, S)
    if pool_device != device or data.num_pages != args.num_pages:
        raise ValueError("pools must lie on the tables' device and hold len(refs) pages")
    n = _pair_lists(src, dst, device)
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        with here:
            workspace = _workspace(args.num_pages, n, workspace, device)
            missing = torch.empty(1, dtype=torch.int32, device=device)
        rc = fa2.library().fa2_pages_fork(ctypes.byref(args), ctypes.byref(data), src.data_ptr(), dst.data_ptr(), n,
                                          missing.data_ptr(), workspace.data_ptr(), _size(workspace), handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_pages_fork")
    return missing


def pages_free(page_table, lens, refs, seqs, page_size: int = 16, stream=None):
    """Empty the sequences ``seqs`` int32 [n]; pages nobody names any more become free (fa2_pages_free)."""
    args, device = _tables(page_table, lens, refs, page_size)
    n = seqs.shape[0] if seqs.dim() == 1 else -1
    _ints("seqs", seqs, (n,), device)
    with fa2._on_device(device):
        handle, _ = _on_stream(stream, device)
        rc = fa2.library().fa2_pages_free(ctypes.byref(args), seqs.data_ptr(), n, handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_pages_free")


def pages_compact(page_table, lens, refs, pools, workspace=None, stream=None):
    """Move the pages in use to the lowest numbers (fa2_pages_compact).

    Page data, ``page_table`` and ``refs`` follow.  Returns int32 [P]: where
    each page went (its own number where it stayed, -1 for a free one).
    """
    import torch

    data, array, S, pool_device = _pools(pools)
    args, device = _tables(page_table, lens, refs, S)
    if pool_device != device or data.num_pages != args.num_pages:
        raise ValueError("pools must lie on the tables' device and hold len(refs) pages")
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        with here:
            workspace = _workspace(args.num_pages, 0, workspace, device)
            moved = torch.empty(args.num_pages, dtype=torch.int32, device=device)
        rc = fa2.library().fa2_pages_compact(ctypes.byref(args), ctypes.byref(data), moved.data_ptr(),
                                             workspace.data_ptr(), _size(workspace), handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_pages_compact")
    return moved


def pages_copy(pools, src, dst, workspace=None, stream=None):
    """Copy pages ``src`` to pages ``dst``, int32 [n], in every plane of ``pools`` (fa2_pages_copy).

    Of several pairs with one destination the last counts; a pair whose source
    is another's destination is skipped and reported (``FA2_ERR_PAGE``).
    """
    data, array, _, device = _pools(pools)
    n = _pair_lists(src, dst, device)
    with fa2._on_device(device):
        handle, here = _on_stream(stream, device)
        with here:
            workspace = _workspace(0, n, workspace, device)
        rc = fa2.library().fa2_pages_copy(ctypes.byref(data), src.data_ptr(), dst.data_ptr(), n,
                                          workspace.data_ptr(), _size(workspace), handle)
    if rc != fa2.FA2_OK:
        raise fa2.FA2Error(rc, "fa2_pages_copy")

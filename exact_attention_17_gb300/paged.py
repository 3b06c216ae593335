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
workspaces that a call makes belong to the stream that it runs on.  A call on the
current device and stream that leaves its outputs to be made goes through the
compiled binding (csrc/binding.cpp), which makes the same checks; whatever that
does not take comes here, and everything where the binding is not built (a call
then costs the host about 40 us instead of 5).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import exact_attention_17_gb300 as fa2

from .build import BINDING_PATH

_LL2, _LL3 = ctypes.c_longlong * 2, ctypes.c_longlong * 3

# Filled by the first call: importing the package does not import torch.
torch = None
_lib = None
_fast = None           # the compiled binding, None where it is not built
_codes = None          # element type -> FA2_DTYPE_*
_raw_stream = None     # device index -> handle of the current stream


def _load():
    global torch, _lib, _fast, _codes, _raw_stream
    import torch as t

    _lib = fa2.library()
    if os.path.exists(BINDING_PATH):
        from . import _binding

        _binding.init(*(ctypes.cast(getattr(_lib, name), ctypes.c_void_p).value for name in (
            "fa2_forward_paged", "fa2_forward_paged_workspace_bytes", "fa2_rope", "fa2_append_paged",
            "fa2_pages_workspace_bytes", "fa2_pages_reserve", "fa2_pages_fork", "fa2_pages_free", "fa2_pages_compact",
            "fa2_pages_copy", "fa2_append_paged_norm", "fa2_norm_rope", "fa2_norm_rope_backward",
            "fa2_norm_rope_backward_workspace_bytes", "fa2_forward_paged_window", "fa2_forward_paged_prefix",
            "fa2_forward_paged_prefix_workspace_bytes", "fa2_forward_window", "fa2_backward_window",
            "fa2_backward_window_workspace_bytes")))
        _fast = _binding
    _codes = fa2._dtype_codes()
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (lambda i: t.cuda.current_stream(i).cuda_stream)
    torch = t


class _Call:
    """The device and the stream of a call.

    ``handle`` is the raw stream.  Within the context the device is current, and
    what torch allocates belongs to that stream (memory that its earlier work
    still uses is not handed out to it, nor its own to others while it runs).
    """

    __slots__ = ("handle", "contexts")

    def __init__(self, device, stream):
        index = device.index
        self.contexts = ()
        if stream is None:
            self.handle = _raw_stream(index)
        else:
            self.handle = handle = getattr(stream, "cuda_stream", stream)
            if handle != _raw_stream(index):
                if handle == 0:
                    on = torch.cuda.default_stream(device)
                else:
                    on = torch.cuda.ExternalStream(handle, device=device)
                self.contexts = (torch.cuda.stream(on),)
        if torch.cuda.current_device() != index:
            self.contexts = (torch.cuda.device(device),) + self.contexts

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self.handle

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _fail(rc, where):
    raise fa2.FA2Error(rc, where)


def _answer(r, where):
    """What the compiled binding answered: the outputs, or a status."""
    if type(r) is int:
        _fail(r, where)
    return r


def _sizes(*sizes):
    """Sizes that go to the library as C ints: ctypes would keep the low 32 bits of larger ones."""
    for n in sizes:
        if not -1 << 31 <= n < 1 << 31:
            raise ValueError(f"a size of {n} does not fit the library's 32-bit integers")


def _ints(name, t, shape, device):
    """An int32 CUDA tensor of `shape`, rows dense."""
    _sizes(*shape)
    if t.dtype is not torch.int32 or t.shape != shape or t.device != device or (shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a dense int32 tensor of shape {tuple(shape)} on {device}")


def _rows(name, t, shape, dtype, device):
    """A [T, H, d] tensor of the cache's type, last dimension dense; its strides."""
    strides = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.device != device or strides[-1] != 1:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device} with a dense last dimension")
    _sizes(*shape)
    return strides


def _cache_args(k_pages, v_pages, page_table, kv_lens, device, dtype):
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise ValueError("k_pages must be bf16 or fp16")
    shape, strides = k_pages.shape, k_pages.stride()
    if not k_pages.is_cuda or len(shape) != 4 or strides[3] != 1:
        raise ValueError("k_pages must be a 4-D CUDA tensor with a dense last dimension")
    if v_pages.dtype is not dtype or v_pages.shape != shape or v_pages.stride() != strides or v_pages.device != device:
        raise ValueError("v_pages must match k_pages in type, shape, strides and device")
    _sizes(*shape)
    table_shape = page_table.shape
    if len(table_shape) != 2:
        raise ValueError("page_table must be [B, M]")
    B, M = table_shape
    _ints("page_table", page_table, table_shape, device)
    _ints("kv_lens", kv_lens, (B,), device)
    return fa2.PagedCacheArgs(k_pages.data_ptr(), v_pages.data_ptr(), shape[0], shape[1], shape[2], shape[3],
                              strides[0], strides[1], strides[2], _codes[dtype], page_table.data_ptr(),
                              page_table.stride(0), M, B, kv_lens.data_ptr())


def _offsets(cu_q, B, T, device):
    """Pointer of cu_q, or None."""
    if cu_q is not None:
        _ints("cu_q", cu_q, (B + 1,), device)
        return cu_q.data_ptr()
    if T != B:
        raise ValueError(f"without cu_q there is one new token for each of the {B} sequences, not {T}")
    return None


@functools.lru_cache(maxsize=1024)
def _paged_workspace_bytes(device_index, *sizes):
    with torch.cuda.device(device_index):
        return _lib.fa2_forward_paged_workspace_bytes(*sizes)


@functools.lru_cache(maxsize=None)
def _default_scale(d):
    """1/sqrt(d) rounded once to float32."""
    return ctypes.c_float(1.0 / math.sqrt(d)).value


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
    if torch is None:
        _load()
    if (_fast is not None and out is None and lse is None and out_dtype is None and workspace is None
            and stream is None):
        r = _fast.forward_paged(q, k_pages, v_pages, page_table, kv_lens, cu_q, causal, scale)
        if r is not None:
            return _answer(r, "fa2_forward_paged")
    return _attend("fa2_forward_paged", (1 if causal else 0,), _paged_workspace_bytes, (), q, k_pages, v_pages, page_table,
                   kv_lens, cu_q, scale, out, lse, out_dtype, workspace, stream)


def _attend(name, own, workspace_bytes, workspace_sizes, q, k_pages, v_pages, page_table, kv_lens, cu_q, scale, out, lse,
            out_dtype, workspace, stream):
    """One of the attention calls over a cache: ``own`` are its arguments between Hq and scale, ``workspace_sizes``
    those of its workspace behind B."""
    dtype, device = k_pages.dtype, k_pages.device
    args = _cache_args(k_pages, v_pages, page_table, kv_lens, device, dtype)
    shape = q.shape
    if len(shape) != 3 or shape[2] != args.d:
        raise ValueError(f"q must be [T, Hq, {args.d}]")
    T, Hq, d = shape
    strides = _rows("q", q, shape, dtype, device)
    if args.kv_heads == 0 or Hq % args.kv_heads != 0:
        raise ValueError(f"{Hq} query heads are no multiple of {args.kv_heads} key/value heads")
    offsets = _offsets(cu_q, args.B, T, device)
    if out_dtype is None:
        out_dtype = dtype
    elif out_dtype is not torch.float32 and out_dtype is not dtype:
        raise ValueError("out_dtype must be fp32 or the cache's type")
    if scale is None:
        scale = _default_scale(d)
    with _Call(device, stream) as handle:
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device=device)
        elif out.dtype is not out_dtype or out.shape != shape or not out.is_contiguous() or out.device != device:
            raise ValueError(f"out must be a contiguous {out_dtype} tensor of shape {(T, Hq, d)} on {device}")
        if lse is None:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=device)
        elif (lse.dtype is not torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()
              or lse.device != device):
            raise ValueError(f"lse must be a contiguous fp32 tensor of shape {(T, Hq)} on {device}")
        if workspace is None:
            size = workspace_bytes(device.index, args.B, *workspace_sizes, T, Hq, args.kv_heads, d, offsets is not None)
            workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=device)
        else:
            size = _workspace_size(workspace, device)
        rc = getattr(_lib, name)(ctypes.byref(args), q.data_ptr(), strides[0], strides[1], out.data_ptr(),
                                 lse.data_ptr(), offsets, T, Hq, *own, scale, _codes[out_dtype], workspace.data_ptr(),
                                 size, handle)
    if rc:
        _fail(rc, name)
    return out, lse


def forward_paged_window(q, k_pages, v_pages, page_table, kv_lens, window: int, sinks: int = 0, cu_q=None,
                         scale: float | None = None, out=None, lse=None, out_dtype=None, workspace=None, stream=None):
    """``forward_paged`` (causal) with a window (fa2_forward_paged_window).

    A token at position p sees the keys j <= p with p - j < window (its own among
    them) or j < sinks.  Pages that no new token sees are not read, nor their
    table entries: they may have been freed.  The other arguments and the
    workspace are ``forward_paged``'s.
    """
    if torch is None:
        _load()
    # a window or sinks beyond every length are all of them
    window, sinks = min(int(window), (1 << 31) - 1), min(int(sinks), (1 << 31) - 1)
    if window < 1 or sinks < 0:
        raise ValueError("window must be at least 1, sinks not negative")
    if (_fast is not None and out is None and lse is None and out_dtype is None and workspace is None
            and stream is None):
        r = _fast.forward_paged_window(q, k_pages, v_pages, page_table, kv_lens, cu_q, window, sinks, scale)
        if r is not None:
            return _answer(r, "fa2_forward_paged_window")
    return _attend("fa2_forward_paged_window", (window, sinks), _paged_workspace_bytes, (), q, k_pages, v_pages,
                   page_table, kv_lens, cu_q, scale, out, lse, out_dtype, workspace, stream)


@functools.lru_cache(maxsize=1024)
def _prefix_workspace_bytes(device_index, *sizes):
    with torch.cuda.device(device_index):
        return _lib.fa2_forward_paged_prefix_workspace_bytes(*sizes)


def forward_paged_prefix(q, k_pages, v_pages, page_table, kv_lens, cu_groups, prefix_lens, cu_q=None,
                         causal: bool = True, scale: float | None = None, out=None, lse=None, out_dtype=None,
                         workspace=None, stream=None):
    """``forward_paged`` for sequences that share prefixes (fa2_forward_paged_prefix).

    Group g is the sequences ``cu_groups[g]`` .. ``cu_groups[g + 1]`` - 1 (int32
    [groups + 1]); their first ``prefix_lens[g]`` tokens (int32 [groups]) lie in
    the same pages, as ``pages_fork`` leaves them, before all new tokens.  Their keys
    are read once for the group.  The part of a prefix behind its last whole
    page is read from each sequence's own pages.  The other arguments are
    ``forward_paged``'s; so are the results, but for the order of the sums.

    It pays for single tokens and short chunks (up to about 80 rows a sequence: new
    tokens times the query heads of a key/value head) where ``forward_paged`` on the same
    table would read more than 200 MB of a group's keys and values again (32 single tokens behind
    8192 with 8 key/value heads of 128: 36 us instead of 110; 8 behind 2000: 22 instead of 19).
    Longer chunks, a prompt's among them, are faster in ``forward_paged``.
    """
    if torch is None:
        _load()
    if (_fast is not None and out is None and lse is None and out_dtype is None and workspace is None
            and stream is None):
        r = _fast.forward_paged_prefix(q, k_pages, v_pages, page_table, kv_lens, cu_q, cu_groups, prefix_lens, causal,
                                       scale)
        if r is not None:
            return _answer(r, "fa2_forward_paged_prefix")
    device = k_pages.device
    if prefix_lens.dim() != 1:
        raise ValueError("prefix_lens must be 1-D")
    groups = prefix_lens.shape[0]
    _ints("prefix_lens", prefix_lens, (groups,), device)
    _ints("cu_groups", cu_groups, (groups + 1,), device)
    own = (cu_groups.data_ptr(), prefix_lens.data_ptr(), groups, 1 if causal else 0)
    return _attend("fa2_forward_paged_prefix", own, _prefix_workspace_bytes if groups else _paged_workspace_bytes,
                   (groups,) if groups else (), q, k_pages, v_pages, page_table, kv_lens, cu_q, scale, out, lse, out_dtype,
                   workspace, stream)


def _workspace_size(workspace, device):
    if not workspace.is_contiguous() or workspace.device != device:
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.numel() * workspace.element_size()


def _inv_freq_args(inv_freq, device, d):
    if inv_freq is None:
        return None, 0
    shape = inv_freq.shape
    if inv_freq.dtype is not torch.float64 or len(shape) != 1 or not inv_freq.is_contiguous() or inv_freq.device != device:
        raise ValueError(f"inv_freq must be a contiguous 1-D float64 tensor on {device}")
    if 2 * shape[0] > d:
        raise ValueError(f"inv_freq holds more than the {d // 2} pairs of a head")
    return inv_freq.data_ptr(), 2 * shape[0]


def append_paged(k, v, k_pages, v_pages, page_table, kv_lens, cu_q=None, q=None, q_out=None, inv_freq=None,
                 interleaved: bool = False, mscale: float = 1.0, stream=None, q_weight=None, k_weight=None,
                 eps: float = 1e-6):
    """Write new tokens into a paged cache (fa2_append_paged, fa2_append_paged_norm).

    k, v [T, Hkv, d] go to their sequences' pages at positions kv_lens[b] - c_b
    + i (the pages must be there: ``pages_reserve``), k rotated at its position
    when ``inv_freq`` is given (see ``rope``).  With ``q`` [T, Hq, d] the
    queries are rotated in the same launch and returned (``q_out``; pass
    ``q_out=q`` to rotate in place).  Rows behind cu_q[B] are not touched.

    ``q_weight`` and ``k_weight`` [d] (both of the cache's type, or both fp32) norm
    each query's and key's row before it is rotated, as ``norm_rope`` does with
    ``eps``; either may be None.
    """
    if torch is None:
        _load()
    if _fast is not None and q is not None and q_out is None and stream is None:
        r = _fast.append_paged(k, v, k_pages, v_pages, page_table, kv_lens, cu_q, q, inv_freq, interleaved, mscale,
                               q_weight, k_weight, eps)
        if r is not None:
            return _answer(r, "fa2_append_paged")
    dtype, device = k_pages.dtype, k_pages.device
    args = _cache_args(k_pages, v_pages, page_table, kv_lens, device, dtype)
    d = args.d
    if k.dim() != 3:
        raise ValueError(f"k must be [T, {args.kv_heads}, {d}]")
    T = k.shape[0]
    shape = (T, args.kv_heads, d)
    ks = _rows("k", k, shape, dtype, device)
    vs = _rows("v", v, shape, dtype, device)
    offsets = _offsets(cu_q, args.B, T, device)
    freq, rotary_dim = _inv_freq_args(inv_freq, device, d)
    normed = q_weight is not None or k_weight is not None
    if normed:
        if q_weight is not None and q is None:
            raise ValueError("q_weight without q")
        if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
            raise ValueError("q_weight and k_weight must have the same type")
        q_norm, _ = _weight_args("q_weight", q_weight, d, dtype, device)
        k_norm, _ = _weight_args("k_weight", k_weight, d, dtype, device)
        code = _codes[(k_weight if q_weight is None else q_weight).dtype]
    with _Call(device, stream) as handle:
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
            Hq, queries, queries_out, qs, qos = 0, None, None, None, None
        else:
            if q.dim() != 3:
                raise ValueError(f"q must be [{T}, Hq, {d}]")
            Hq = q.shape[1]
            st = _rows("q", q, (T, Hq, d), dtype, device)
            if q_out is None:
                q_out = torch.empty((T, Hq, d), dtype=dtype, device=device)
            so = _rows("q_out", q_out, (T, Hq, d), dtype, device)
            queries, queries_out = q.data_ptr(), q_out.data_ptr()
            qs, qos = _LL2(st[0], st[1]), _LL2(so[0], so[1])
        arrays = (ctypes.byref(args), k.data_ptr(), _LL2(ks[0], ks[1]), v.data_ptr(), _LL2(vs[0], vs[1]), queries, qs,
                  queries_out, qos, Hq, offsets, T)
        rotary = (freq, rotary_dim, 1 if interleaved else 0, mscale, handle)
        if normed:
            rc = _lib.fa2_append_paged_norm(*arrays, q_norm, k_norm, code, eps, *rotary)
        else:
            rc = _lib.fa2_append_paged(*arrays, *rotary)
    if rc:
        _fail(rc, "fa2_append_paged_norm" if normed else "fa2_append_paged")
    return q_out


def _weight_args(name, weight, d, dtype, device):
    """Pointer of a norm's weights (None for none) and the code of their type."""
    if weight is None:
        return None, None
    if ((weight.dtype is not dtype and weight.dtype is not torch.float32) or weight.shape != (d,)
            or not weight.is_contiguous() or weight.device != device):
        raise ValueError(f"{name} must be a contiguous {dtype} or fp32 tensor of shape {(d,)} on {device}")
    return weight.data_ptr(), _codes[weight.dtype]


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
    if torch is None:
        _load()
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


def _strides3(t):
    """Strides {batch, head, token} of [B, H, N, d], or of packed [T, H, d]: one batch, tokens outside the heads."""
    s = t.stride()
    return _LL3(s[0], s[1], s[2]) if len(s) == 4 else _LL3(0, s[1], s[0])


def _heads(name, x):
    """Rows of heads, [B, H, N, d] or [T, H, d]: their sizes B, H, N, d and strides."""
    dim = x.dim()
    if x.dtype not in _codes or not x.is_cuda or (dim != 4 and dim != 3) or x.stride(-1) != 1:
        raise ValueError(f"{name} must be a bf16, fp16 or fp32 CUDA tensor [T, H, d] or [B, H, N, d], last dimension dense")
    _sizes(*x.shape)
    if dim == 3:
        N, H, d = x.shape
        return 1, H, N, d, _strides3(x)
    return (*x.shape, _strides3(x))


def _like(name, t, x):
    """Strides of an array that must match x in type, shape and device, last dimension dense."""
    if t.dtype is not x.dtype or t.shape != x.shape or t.device != x.device or t.stride(-1) != 1:
        raise ValueError(f"{name} must be a {x.dtype} tensor of shape {tuple(x.shape)} on {x.device}, last dimension dense")
    return _strides3(t)


def _position_args(positions, B, N, dim, device):
    """Positions' pointer, whether they are 64-bit, and the stride of a batch."""
    ps = positions.shape
    if positions.device != device or (positions.dtype is not torch.int32 and positions.dtype is not torch.int64):
        raise ValueError(f"positions must be int32 or int64 on {device}")
    if (ps != (N,) and ps != (B, N)) or (N > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions must be a dense [{N}]" + (f" or [{B}, {N}]" if dim == 4 else ""))
    return positions.data_ptr(), 1 if positions.dtype is torch.int64 else 0, positions.stride(0) if len(ps) == 2 else 0


def _rope(x, positions, inv_freq, interleaved, mscale, out, stream, transposed):
    if torch is None:
        _load()
    if _fast is not None and out is None and stream is None:
        r = _fast.rope(x, positions, inv_freq, interleaved, mscale, transposed)
        if r is not None:
            return _answer(r, "fa2_rope")
    B, H, N, d, xs = _heads("x", x)
    dtype, device, shape = x.dtype, x.device, x.shape
    place = _position_args(positions, B, N, len(shape), device)
    freq, rotary_dim = _inv_freq_args(inv_freq, device, d)
    with _Call(device, stream) as handle:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        ys = _like("out", out, x)
        rc = _lib.fa2_rope(x.data_ptr(), xs, out.data_ptr(), ys, B, H, N, d, *place, freq, rotary_dim,
                           1 if interleaved else 0, mscale, transposed, _codes[dtype], handle)
    if rc:
        _fail(rc, "fa2_rope")
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
    return _rope(x, positions, inv_freq, interleaved, mscale, out, stream, 0)


def rope_backward(do, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0, out=None, stream=None):
    """Gradient of ``rope`` with respect to x for the upstream gradient ``do``
    (the transposed rotation); arguments as ``rope``."""
    return _rope(do, positions, inv_freq, interleaved, mscale, out, stream, 1)


def _tables(page_table, lens, refs, page_size):
    if torch is None:
        _load()
    device, shape, pages = page_table.device, page_table.shape, refs.shape
    if len(shape) != 2 or not page_table.is_cuda or len(pages) != 1:
        raise ValueError("page_table must be a CUDA tensor [B, M], refs [P]")
    B, M = shape
    _ints("page_table", page_table, shape, device)
    _ints("lens", lens, (B,), device)
    _ints("refs", refs, pages, device)
    _sizes(page_size)
    return fa2.PageTablesArgs(page_table.data_ptr(), page_table.stride(0), M, B, lens.data_ptr(), refs.data_ptr(),
                              pages[0], page_size), device


def _pools(pools):
    """Page data as an array of planes: a tensor [..., P, Hkv, S, d], or a list of such tensors.

    (arguments of the library, the array they point to, slots per page, device)
    """
    if torch is None:
        _load()
    tensors = (pools,) if torch.is_tensor(pools) else tuple(pools)
    if not tensors:
        raise ValueError("pools must hold at least one tensor")
    first, pointers = tensors[0], []
    device, dtype, size = first.device, first.dtype, first.element_size()
    for t in tensors:
        shape, strides = t.shape, t.stride()
        if not t.is_cuda or len(shape) < 4:
            raise ValueError("pools must be CUDA tensors [..., P, Hkv, S, d]")
        if t is not first and (shape[-4:] != first.shape[-4:] or strides[-4:] != first.stride()[-4:]
                               or t.dtype is not dtype or t.device != device):
            raise ValueError("all pools must have the same pages, strides, type and device")
        planes = [t.data_ptr()]
        for n, st in zip(shape[:-4], strides[:-4]):   # the leading dimensions, outermost first
            planes = [p + i * st * size for p in planes for i in range(n)]
        pointers += planes
    P, Hkv, S, d = first.shape[-4:]
    _sizes(P, Hkv, S, d)
    strides = first.stride()
    if strides[-1] != 1 or strides[-2] != d or strides[-3] != S * d:
        dense = 1   # in another order, perhaps
        for st, n in sorted(zip(strides[-3:], (Hkv, S, d))):
            if n > 1 and st != dense:
                raise ValueError("the elements of a page must be dense")
            dense *= n
    array = (ctypes.c_void_p * max(len(pointers), 1))(*pointers)
    args = fa2.PagePoolsArgs(ctypes.addressof(array), len(pointers), P, strides[-4] * size, Hkv * S * d * size)
    return args, array, S, device


@functools.lru_cache(maxsize=1024)
def _pages_workspace_bytes(num_pages, n):
    return max(_lib.fa2_pages_workspace_bytes(num_pages, n), 1)


def _workspace(num_pages, n, given, device):
    """(workspace, bytes)"""
    if given is None:
        size = _pages_workspace_bytes(num_pages, n)
        return torch.empty(size, dtype=torch.uint8, device=device), size
    return given, _workspace_size(given, device)


def _list(name, t, device):
    """Length of a 1-D int32 tensor."""
    shape = t.shape
    if len(shape) != 1:
        raise ValueError(f"{name} must be 1-D")
    _ints(name, t, shape, device)
    return shape[0]


def pages_reserve(page_table, lens, refs, add, page_size: int, workspace=None, stream=None):
    """Make room for ``add`` int32 [B] more tokens (fa2_pages_reserve).

    ``lens`` grows by ``add`` and ``page_table`` by the pages that takes, the
    free ones (``refs`` [P] == 0) of the lowest numbers.  Returns an int32 CUDA
    tensor [1]: 0, or the number of pages that lack, or -1 where a table row is
    too short -- then nothing has changed.
    """
    if torch is None:
        _load()
    if _fast is not None and workspace is None and stream is None:
        r = _fast.pages_reserve(page_table, lens, refs, add, page_size)
        if r is not None:
            return _answer(r, "fa2_pages_reserve")
    args, device = _tables(page_table, lens, refs, page_size)
    _ints("add", add, (args.B,), device)
    with _Call(device, stream) as handle:
        workspace, size = _workspace(args.num_pages, 0, workspace, device)
        missing = torch.empty(1, dtype=torch.int32, device=device)
        rc = _lib.fa2_pages_reserve(ctypes.byref(args), add.data_ptr(), missing.data_ptr(), workspace.data_ptr(), size,
                                    handle)
    if rc:
        _fail(rc, "fa2_pages_reserve")
    return missing


def pages_fork(page_table, lens, refs, src, dst, pools, workspace=None, stream=None):
    """Sequences ``dst`` (empty) become copies of ``src``, int32 [n] (fa2_pages_fork).

    Full pages are shared, a partly filled last page is copied in every plane of
    ``pools`` (a tensor [..., P, Hkv, S, d] or a list of them: all the layers' K
    and V).  Returns the pages that lack as ``pages_reserve`` does.
    """
    if torch is None:
        _load()
    if _fast is not None and workspace is None and stream is None:
        r = _fast.pages_fork(page_table, lens, refs, src, dst, pools)
        if r is not None:
            return _answer(r, "fa2_pages_fork")
    data, array, S, pool_device = _pools(pools)
    args, device = _tables(page_table, lens, refs, S)
    if pool_device != device or data.num_pages != args.num_pages:
        raise ValueError("pools must lie on the tables' device and hold len(refs) pages")
    n = _list("src", src, device)
    _ints("dst", dst, (n,), device)
    with _Call(device, stream) as handle:
        workspace, size = _workspace(args.num_pages, n, workspace, device)
        missing = torch.empty(1, dtype=torch.int32, device=device)
        rc = _lib.fa2_pages_fork(ctypes.byref(args), ctypes.byref(data), src.data_ptr(), dst.data_ptr(), n,
                                 missing.data_ptr(), workspace.data_ptr(), size, handle)
    if rc:
        _fail(rc, "fa2_pages_fork")
    return missing


def pages_free(page_table, lens, refs, seqs, stream=None):
    """Empty the sequences ``seqs`` int32 [n]; pages nobody names any more become free (fa2_pages_free)."""
    if torch is None:
        _load()
    if _fast is not None and stream is None:
        r = _fast.pages_free(page_table, lens, refs, seqs)
        if r is not None:
            _answer(r, "fa2_pages_free")
            return
    args, device = _tables(page_table, lens, refs, 16)   # (the slots per page play no part)
    n = _list("seqs", seqs, device)
    with _Call(device, stream) as handle:
        rc = _lib.fa2_pages_free(ctypes.byref(args), seqs.data_ptr(), n, handle)
    if rc:
        _fail(rc, "fa2_pages_free")


def pages_compact(page_table, lens, refs, pools, workspace=None, stream=None):
    """Move the pages in use to the lowest numbers (fa2_pages_compact).

    Page data, ``page_table`` and ``refs`` follow.  Returns int32 [P]: where
    each page went (its own number where it stayed, -1 for a free one).
    """
    if torch is None:
        _load()
    if _fast is not None and workspace is None and stream is None:
        r = _fast.pages_compact(page_table, lens, refs, pools)
        if r is not None:
            return _answer(r, "fa2_pages_compact")
    data, array, S, pool_device = _pools(pools)
    args, device = _tables(page_table, lens, refs, S)
    if pool_device != device or data.num_pages != args.num_pages:
        raise ValueError("pools must lie on the tables' device and hold len(refs) pages")
    with _Call(device, stream) as handle:
        workspace, size = _workspace(args.num_pages, 0, workspace, device)
        moved = torch.empty(args.num_pages, dtype=torch.int32, device=device)
        rc = _lib.fa2_pages_compact(ctypes.byref(args), ctypes.byref(data), moved.data_ptr(), workspace.data_ptr(),
                                    size, handle)
    if rc:
        _fail(rc, "fa2_pages_compact")
    return moved


def pages_copy(pools, src, dst, workspace=None, stream=None):
    """Copy pages ``src`` to pages ``dst``, int32 [n], in every plane of ``pools`` (fa2_pages_copy).

    Of several pairs with one destination the last counts; a pair whose source
    is another's destination is skipped and reported (``FA2_ERR_PAGE``).
    """
    if torch is None:
        _load()
    if _fast is not None and workspace is None and stream is None:
        r = _fast.pages_copy(pools, src, dst)
        if r is not None:
            _answer(r, "fa2_pages_copy")
            return
    data, array, _, device = _pools(pools)
    n = _list("src", src, device)
    _ints("dst", dst, (n,), device)
    with _Call(device, stream) as handle:
        workspace, size = _workspace(0, n, workspace, device)
        rc = _lib.fa2_pages_copy(ctypes.byref(data), src.data_ptr(), dst.data_ptr(), n, workspace.data_ptr(), size,
                                 handle)
    if rc:
        _fail(rc, "fa2_pages_copy")

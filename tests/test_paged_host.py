"""The paged-cache entry points refuse bad arguments on the host, before any GPU work."""
import ctypes

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return fa2.library()


def cache(**kw):
    a = dict(k_pages=16, v_pages=16, num_pages=4, kv_heads=2, page_size=16, d=64, page_stride=2048, head_stride=1024,
             slot_stride=64, dtype=fa2.FA2_DTYPE_BF16, page_table=16, table_stride=3, table_width=3, B=2, kv_lens=16)
    a.update(kw)
    return fa2.PagedCacheArgs(**a)


BAD_CACHES = [
    (dict(dtype=fa2.FA2_DTYPE_FP32), "DTYPE"), (dict(num_pages=0), "SHAPE"), (dict(kv_heads=0), "SHAPE"),
    (dict(B=-1), "SHAPE"), (dict(table_width=0), "SHAPE"), (dict(page_size=8), "SHAPE"), (dict(page_size=48), "SHAPE"),
    (dict(page_size=2048), "SHAPE"), (dict(table_width=1 << 27), "SHAPE"), (dict(d=96), "HEADDIM"),
    (dict(slot_stride=32), "SHAPE"), (dict(head_stride=0), "SHAPE"), (dict(page_stride=8), "SHAPE"),
    (dict(page_stride=1 << 40), "SHAPE"), (dict(table_stride=2), "SHAPE"), (dict(k_pages=None), "NULL"),
    (dict(v_pages=None), "NULL"), (dict(page_table=None), "NULL"), (dict(kv_lens=None), "NULL"),
    (dict(k_pages=24), "ALIGN"), (dict(v_pages=8), "ALIGN"), (dict(slot_stride=68), "ALIGN"),
    (dict(head_stride=1028), "ALIGN"), (dict(page_stride=2049), "ALIGN"), (dict(page_table=18), "ALIGN"),
    (dict(kv_lens=2), "ALIGN"),
]


def forward(c, Q=16, qt=256, qh=64, O=16, LSE=16, cu=None, T=2, Hq=4, causal=1, scale=0.125,
            o_dtype=fa2.FA2_DTYPE_BF16, ws=256, size=1 << 30):
    return fa2.library().fa2_forward_paged(None if c is None else ctypes.byref(c), Q, qt, qh, O, LSE, cu, T, Hq,
                                           causal, scale, o_dtype, ws, size, None)


def test_forward_paged(lib):
    for bad, code in BAD_CACHES:
        assert forward(cache(**bad)) == getattr(fa2, "FA2_ERR_" + code), bad
    c = cache()
    assert forward(None) == fa2.FA2_ERR_NULL
    # empty problems launch nothing
    assert forward(c, T=0, Q=None) == fa2.FA2_OK
    assert forward(c, Hq=0) == fa2.FA2_OK
    assert forward(cache(B=0)) == fa2.FA2_OK
    assert forward(c, T=-1) == fa2.FA2_ERR_SHAPE
    assert forward(c, Hq=-4) == fa2.FA2_ERR_SHAPE
    assert forward(c, Hq=3) == fa2.FA2_ERR_SHAPE            # no multiple of the key/value heads
    assert forward(c, Hq=258) == fa2.FA2_ERR_SHAPE          # a group of 129
    assert forward(c, T=3) == fa2.FA2_ERR_SHAPE             # without offsets T is B
    assert forward(c, qt=32) == fa2.FA2_ERR_SHAPE
    assert forward(c, qh=32) == fa2.FA2_ERR_SHAPE
    assert forward(c, qt=1 << 40) == fa2.FA2_ERR_SHAPE
    for dt in (fa2.FA2_DTYPE_FP16, 7):
        assert forward(c, o_dtype=dt) == fa2.FA2_ERR_DTYPE
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert forward(c, scale=s) == fa2.FA2_ERR_SCALE
    for name in ("Q", "O", "LSE", "ws"):
        assert forward(c, **{name: None}) == fa2.FA2_ERR_NULL
    for name, value in (("Q", 8), ("O", 8), ("LSE", 2), ("ws", 128), ("cu", 2), ("qt", 260), ("qh", 68)):
        assert forward(c, **{name: value}) == fa2.FA2_ERR_ALIGN, name


def test_forward_paged_workspace(lib):
    f = lib.fa2_forward_paged_workspace_bytes
    for bad in ((0, 4, 8, 2, 64, 0), (2, 0, 8, 2, 64, 0), (2, 2, 0, 2, 64, 0), (2, 2, 7, 2, 64, 0), (2, 2, 8, 2, 96, 0),
                (2, 2, 258, 2, 64, 0)):
        assert f(*bad) == 0


def rope(X=16, xs=(0, 64, 64), Y=4096, ys=(0, 64, 64), B=1, H=1, N=4, d=64, pos=16, pos64=0, ps=0, freq=16, r=64,
         inter=0, m=1.0, dtype=fa2.FA2_DTYPE_BF16):
    s = lambda t: None if t is None else (ctypes.c_longlong * 3)(*t)  # noqa: E731
    return fa2.library().fa2_rope(X, s(xs), Y, s(ys), B, H, N, d, pos, pos64, ps, freq, r, inter, m, 0, dtype, None)


def test_rope(lib):
    for empty in (dict(B=0), dict(H=0), dict(N=0, X=None)):
        assert rope(**empty) == fa2.FA2_OK
    for bad in (dict(B=-1), dict(N=-1), dict(d=0), dict(r=66), dict(r=3), dict(r=-2), dict(xs=(0, 64, -64)),
                dict(ys=(0, 64, 0)), dict(ys=(0, 64, 32)), dict(B=2, ys=(256, 64, 64), ps=-1)):
        assert rope(**bad) == fa2.FA2_ERR_SHAPE, bad
    for d in (63, 1026):
        assert rope(d=d, r=2) == fa2.FA2_ERR_HEADDIM
    assert rope(dtype=5) == fa2.FA2_ERR_DTYPE
    for m in (float("inf"), float("nan")):
        assert rope(m=m) == fa2.FA2_ERR_SCALE
    for bad in (dict(X=None), dict(Y=None), dict(pos=None), dict(freq=None), dict(xs=None), dict(ys=None)):
        assert rope(**bad) == fa2.FA2_ERR_NULL, bad
    for bad in (dict(X=17), dict(Y=4097), dict(pos=2), dict(pos=4, pos64=1), dict(freq=4),
                dict(X=18, inter=1), dict(ys=(0, 64, 65), inter=1)):
        assert rope(**bad) == fa2.FA2_ERR_ALIGN, bad


def append(c, K=16, ks=(128, 64), V=16, vs=(128, 64), Q=16, qs=(256, 64), Qo=4096, qos=(256, 64), Hq=4, cu=None, T=2,
           freq=16, r=64, m=1.0):
    s = lambda t: None if t is None else (ctypes.c_longlong * 2)(*t)  # noqa: E731
    return fa2.library().fa2_append_paged(None if c is None else ctypes.byref(c), K, s(ks), V, s(vs), Q, s(qs), Qo,
                                          s(qos), Hq, cu, T, freq, r, 0, m, None)


def test_append_paged(lib):
    for bad, code in BAD_CACHES:
        assert append(cache(**bad)) == getattr(fa2, "FA2_ERR_" + code), bad
    c = cache()
    assert append(None) == fa2.FA2_ERR_NULL
    assert append(c, T=0, K=None) == fa2.FA2_OK
    assert append(cache(B=0)) == fa2.FA2_OK
    for bad in (dict(T=-1), dict(T=3), dict(Hq=-1), dict(r=66), dict(r=7), dict(ks=(32, 64)), dict(vs=(128, 8)),
                dict(qs=(256, 8)), dict(qos=(0, 64))):
        assert append(c, **bad) == fa2.FA2_ERR_SHAPE, bad
    for bad in (dict(K=None), dict(V=None), dict(Q=None), dict(Qo=None), dict(ks=None), dict(vs=None), dict(qs=None),
                dict(qos=None), dict(freq=None)):
        assert append(c, **bad) == fa2.FA2_ERR_NULL, bad
    for bad in (dict(K=8), dict(V=8), dict(Q=8), dict(Qo=8), dict(ks=(132, 64)), dict(cu=2), dict(freq=4)):
        assert append(c, **bad) == fa2.FA2_ERR_ALIGN, bad
    assert append(c, m=float("nan")) == fa2.FA2_ERR_SCALE


def tables(**kw):
    a = dict(page_table=16, table_stride=3, table_width=3, B=2, lens=16, refs=16, num_pages=4, page_size=16)
    a.update(kw)
    return fa2.PageTablesArgs(**a)


def pools(planes=(16, 32), **kw):
    a = dict(num_planes=len(planes), num_pages=4, page_stride=1024, page_bytes=512)
    a.update(kw)
    array = (ctypes.c_void_p * max(len(planes), 1))(*planes)
    p = fa2.PagePoolsArgs(ctypes.cast(array, ctypes.c_void_p), **a)
    p.keep = array
    return p


BAD_TABLES = [(dict(B=-1), "SHAPE"), (dict(table_width=0), "SHAPE"), (dict(num_pages=0), "SHAPE"),
              (dict(num_pages=1 << 21), "SHAPE"), (dict(page_size=24), "SHAPE"), (dict(table_stride=2), "SHAPE"),
              (dict(page_table=None), "NULL"), (dict(lens=None), "NULL"), (dict(refs=None), "NULL"),
              (dict(page_table=2), "ALIGN"), (dict(lens=1), "ALIGN"), (dict(refs=2), "ALIGN")]
BAD_POOLS = [(dict(page_bytes=8), "SHAPE"), (dict(page_stride=256), "SHAPE"), (dict(num_planes=257), "SHAPE"),
             (dict(page_bytes=504), "ALIGN"), (dict(page_stride=1032), "ALIGN"), (dict(planes=(16, 8)), "ALIGN"),
             (dict(planes=(16, None)), "NULL")]


def test_pages(lib):
    def ref(x):
        return None if x is None else ctypes.byref(x)

    def reserve(t, add=16, missing=16, ws=256):
        return lib.fa2_pages_reserve(ref(t), add, missing, ws, 1 << 20, None)

    def fork(t, d, src=16, dst=16, n=1, missing=16, ws=256):
        return lib.fa2_pages_fork(ref(t), ref(d), src, dst, n, missing, ws, 1 << 20, None)

    def free(t, seqs=16, n=1):
        return lib.fa2_pages_free(ref(t), seqs, n, None)

    def compact(t, d, moved=16):
        return lib.fa2_pages_compact(ref(t), ref(d), moved, 256, 1 << 20, None)

    def copy(d, src=16, dst=16, n=1):
        return lib.fa2_pages_copy(ref(d), src, dst, n, 256, 1 << 20, None)

    for bad, code in BAD_TABLES:
        code, t = getattr(fa2, "FA2_ERR_" + code), tables(**bad)
        assert [reserve(t), fork(t, pools()), free(t), compact(t, pools())] == [code] * 4, bad
    for bad, code in BAD_POOLS:
        code, d = getattr(fa2, "FA2_ERR_" + code), pools(**bad)
        assert [fork(tables(), d), compact(tables(), d), copy(d)] == [code] * 3, bad
    null, shape = fa2.FA2_ERR_NULL, fa2.FA2_ERR_SHAPE
    assert [reserve(None), fork(None, pools()), fork(tables(), None), free(None), compact(None, pools()),
            compact(tables(), None), copy(None)] == [null] * 7
    assert [reserve(tables(), add=None), reserve(tables(), missing=None), fork(tables(), pools(), src=None),
            fork(tables(), pools(), dst=None), fork(tables(), pools(), missing=None), free(tables(), seqs=None),
            compact(tables(), pools(), moved=None), copy(pools(), src=None), copy(pools(), dst=None)] == [null] * 9
    assert [fork(tables(), pools(), n=-1), fork(tables(), pools(num_pages=5)), free(tables(), n=-1),
            compact(tables(), pools(num_pages=5)), copy(pools(), n=-1), copy(pools(), n=(1 << 16) + 1)] == [shape] * 6
    assert free(tables(), n=0, seqs=None) == fa2.FA2_OK
    assert copy(pools(), n=0, src=None) == fa2.FA2_OK


def test_pages_workspace(lib):
    f = lib.fa2_pages_workspace_bytes
    assert f(0, 0) == 256
    assert f(1000, 5) == (4 * 2001 + 255) // 256 * 256
    assert f(3, 100) == (4 * 301 + 255) // 256 * 256
    assert f(-1, 0) == f(0, -1) == f(1 << 21, 0) == f(0, (1 << 16) + 1) == 0


def test_binding_refuses_host_tensors_and_bad_arguments():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa2.forward_paged(q, k, k, i32(2, 3), i32(2))
    with pytest.raises(ValueError, match="bf16 or fp16"):
        fa2.append_paged(q, q, k.float(), k.float(), i32(2, 3), i32(2))
    with pytest.raises(ValueError, match="CUDA"):
        fa2.rope(q, i32(2), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        fa2.pages_reserve(i32(2, 3), i32(2), i32(4), i32(2), 16)
    with pytest.raises(ValueError, match="CUDA"):
        fa2.pages_copy(k, i32(1), i32(1))
    with pytest.raises(ValueError, match="at least one"):
        fa2.pages_copy([], i32(1), i32(1))
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            fa2.rope_inv_freq(**bad)


def test_status_text():
    assert "cache" in fa2.fa2_status_string(fa2.FA2_ERR_PAGE)

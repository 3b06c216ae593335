"""Arrays that a call writes may not overlap themselves: refused on the host, before any GPU work."""
import ctypes

import pytest

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return fa2.library()


def longs(t):
    return (ctypes.c_longlong * len(t))(*t)


def rope(lib, sizes, ys, xs=None, Y=1 << 20):
    B, H, N = sizes
    xs = (H * N * 64, N * 64, 64) if xs is None else xs
    return lib.fa2_rope(4096, longs(xs), Y, longs(ys), B, H, N, 64, 4096, 0, 0, 4096, 64, 0, 1.0, 0,
                        fa2.FA2_DTYPE_BF16, None)


# sizes [B, H, N] of rows of 64, strides whose rows meet
MEET = [((1, 2, 3), (0, 64, 64)), ((1, 2, 3), (0, 128, 64)), ((2, 1, 3), (64, 0, 64)), ((2, 3, 1), (128, 64, 0)),
        ((2, 3, 4), (64 * 4, 64 * 7, 64)), ((2, 3, 4), (64 * 12, 64, 64 * 2)), ((2, 3, 4), (64 * 11, 64 * 4, 64)),
        ((5, 1, 7), (96, 0, 80))]
# and that do not: dense, transposed, tokens outermost, padded, one batch's strides of no account
APART = [((2, 3, 4), (64 * 12, 64 * 4, 64)), ((2, 3, 4), (64 * 4, 64 * 8, 64)), ((2, 3, 4), (64 * 12, 64, 64 * 3)),
         ((2, 3, 4), (64, 64 * 8, 64 * 2)), ((2, 3, 4), (5000, 400, 72)), ((1, 3, 4), (0, 64, 64 * 3)), ((1, 1, 1), (0, 0, 0))]


def meets(sizes, strides):
    """Two rows of 64 share an element, row against row."""
    at = sorted(b * strides[0] + h * strides[1] + n * strides[2]
                for b in range(sizes[0]) for h in range(sizes[1]) for n in range(sizes[2]))
    return any(y - x < 64 for x, y in zip(at, at[1:]))


def test_the_cases_are_what_they_say():
    assert all(meets(*c) for c in MEET) and not any(meets(*c) for c in APART)


def test_rope(lib):
    for sizes, ys in MEET:
        assert rope(lib, sizes, ys) == fa2.FA2_ERR_SHAPE, (sizes, ys)
        assert rope(lib, sizes, ys, xs=ys, Y=4096) == fa2.FA2_ERR_SHAPE, (sizes, ys)       # in place
    # what is read may: these get past the arguments' checks, to the device's
    fine = rope(lib, (2, 3, 4), (64 * 12, 64 * 4, 64))
    assert fine in (fa2.FA2_ERR_DEVICE, fa2.FA2_ERR_MEMORY)
    for sizes, ys in APART:
        assert rope(lib, sizes, ys) == fine, (sizes, ys)
    assert rope(lib, (2, 3, 4), (64 * 12, 64 * 4, 64), xs=(0, 0, 0)) == fine


def append(lib, pages=(2048, 1024, 64), q_out=(256, 64), T=2, Hq=4, shape=(4, 2, 16)):
    P, H, S = shape
    c = fa2.PagedCacheArgs(k_pages=4096, v_pages=1 << 20, num_pages=P, kv_heads=H, page_size=S, d=64,
                           page_stride=pages[0], head_stride=pages[1], slot_stride=pages[2], dtype=fa2.FA2_DTYPE_BF16,
                           page_table=16, table_stride=3, table_width=3, B=T, kv_lens=16)
    return lib.fa2_append_paged(ctypes.byref(c), 16, longs((128, 64)), 16, longs((128, 64)), 16, longs((256, 64)),
                                1 << 24, longs(q_out), Hq, None, T, None, 0, 0, 1.0, None)


def test_append(lib):
    fine = append(lib)
    assert fine in (fa2.FA2_ERR_DEVICE, fa2.FA2_ERR_MEMORY)
    for q_out in ((64, 64), (128, 64), (64, 72), (192, 64)):
        assert append(lib, q_out=q_out) == fa2.FA2_ERR_SHAPE, q_out
    for q_out in ((64, 128), (264, 64), (72, 144)):
        assert append(lib, q_out=q_out) == fine, q_out
    for pages in ((1024, 1024, 64), (2048, 512, 64), (2048, 64, 64), (1024, 2048, 64), (2040, 1024, 64)):
        assert append(lib, pages=pages) == fa2.FA2_ERR_SHAPE, pages
    for pages in ((2048, 64, 128), (1024, 4096, 64), (64, 4096, 256), (6144, 1024, 64)):
        assert append(lib, pages=pages) == fine, pages
    assert append(lib, pages=(0, 0, 64), shape=(1, 1, 16)) == fine

"""``fa2_check_window_plan``: the forms that windowed calls take, on the host alone."""
import ctypes

import pytest

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return fa2.library()


def plan(B=1, H=4, Hkv=2, Nq=500, Nk=500, d=128, window=100, sinks=0, sms=152):
    out = (ctypes.c_int * 4)()
    rc = fa2.library().fa2_check_window_plan(B, H, Hkv, Nq, Nk, d, window, sinks, sms, out)
    return rc, list(out)


def test_refusals():
    for bad in (dict(B=0), dict(H=0, Hkv=0), dict(Nq=0), dict(Nk=0), dict(window=0), dict(sinks=-1), dict(H=3),
                dict(sms=0), dict(sms=-5)):
        assert plan(**bad) == (fa2.FA2_ERR_SHAPE, [0] * 4), bad
    assert plan(d=96)[0] == fa2.FA2_ERR_HEADDIM
    assert fa2.library().fa2_check_window_plan(1, 4, 2, 500, 500, 128, 100, 0, 152, None) == fa2.FA2_ERR_NULL


def test_two_sub_tiles_for_long_windows_of_many_blocks():
    long = dict(B=2, H=40, Hkv=8, Nq=1100, Nk=1100, d=128, window=1050)
    assert plan(**long)[1][0] == 2
    for change in (dict(window=1024), dict(B=1), dict(Nq=128), dict(d=256), dict(d=64)):
        assert plan(**{**long, **change})[1][0] == 1, change
    assert plan(B=2, H=20, Hkv=4, Nq=4300, Nk=4300, d=64, window=4200)[1][0] == 2
    assert plan(B=2, H=20, Hkv=4, Nq=4300, Nk=4300, d=64, window=4096)[1][0] == 1

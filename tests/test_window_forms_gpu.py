"""The windowed forward pass with two query sub-tiles a CTA, which it takes by its sizes: ``fa2_check_window_plan`` says
whether a call does."""
import ctypes

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import release_memory
from test_window_gpu import BF, HF, check_forward, inputs

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


def plan(B, H, Hkv, Nq, Nk, d, window, sinks):
    out = (ctypes.c_int * 4)()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert fa2.library().fa2_check_window_plan(B, H, Hkv, Nq, Nk, d, window, sinks, sms, out) == fa2.FA2_OK
    return dict(zip(("sub_tiles", "group", "parts", "sink_parts"), out))


def name(c):
    return f"{str(c[0])[6:]}-{c[1]}x{c[2]}.{c[3]}x{c[4]}.{c[5]}x{c[6]}-w{c[7]}-s{c[8]}"


TWO = [
    # dtype, B, H, Hkv, Nq, Nk, d, window, sinks
    (BF, 2, 40, 8, 1100, 1100, 128, 1050, 0),       # the last block's second sub-tile has no rows
    (HF, 2, 40, 8, 1100, 1100, 128, 1050, 4),
    (BF, 2, 40, 40, 1200, 1200, 128, 1030, 130),    # it has some
    (BF, 2, 40, 10, 1600, 300, 128, 1100, 0),       # late rows without a key, whole blocks of them
    (HF, 2, 40, 10, 1600, 300, 128, 1100, 2),
    (BF, 2, 40, 8, 1100, 2000, 128, 1026, 1500),    # more keys than queries, sinks of everything
    (BF, 2, 40, 8, 1280, 1280, 128, 5000, 0),       # the window holds everything
    (BF, 1, 18, 6, 4300, 4300, 64, 4200, 0),
    (HF, 1, 18, 18, 4300, 4300, 64, 4100, 70),
    (BF, 1, 20, 5, 4230, 90, 64, 4110, 3),
]


@pytest.mark.parametrize("case", TWO, ids=name)
def test_two_sub_tiles(case):
    dtype, B, H, Hkv, Nq, Nk, d, window, sinks = case
    assert plan(*case[1:])["sub_tiles"] == 2
    q, k, v = inputs(dtype, B, H, Hkv, Nq, Nk, d)
    check_forward(q, k, v, window, sinks)
    check_forward(q, k, v, window, sinks, out_dtype=dtype)

"""Gradients of windows whose heads run in several groups, the last of them shorter, and whose key blocks are cut into
items, all of them or those with sinks alone."""
import math

import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild
from paged_reference import EPS, release_memory
from test_window_forms_gpu import name, plan
from test_window_gpu import BF, F32, HF, close, inputs, normal
from window_reference import backward, seen

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


GROUPS = [
    # (dtype, B, H, Hkv, Nq, Nk, d, window, sinks), groups' heads, items of a block without sinks and of one with: several?
    ((BF, 2, 48, 6, 600, 600, 128, 300, 0), [4, 4, 4], True, None),
    ((HF, 1, 56, 7, 600, 600, 128, 300, 0), [4, 3], True, None),        # a shorter last group
    ((BF, 1, 56, 7, 600, 600, 128, 300, 4), [4, 3], True, True),
    ((HF, 1, 40, 5, 600, 600, 128, 300, 200), [4, 1], True, True),
    ((BF, 3, 76, 19, 300, 300, 128, 100, 4), [29, 28], False, True),    # blocks with sinks alone in several items
    ((BF, 3, 76, 19, 300, 300, 128, 100, 0), [29, 28], False, None),
    ((BF, 1, 56, 7, 500, 200, 128, 300, 130), [4, 3], True, True),      # fewer keys, late rows without one but sinks
    ((HF, 1, 56, 7, 200, 700, 128, 150, 0), [4, 3], True, None),        # keys behind the last query
    ((HF, 1, 112, 7, 600, 600, 64, 300, 4), [4, 3], True, True),
]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("case, groups, cut, sinks_cut", GROUPS, ids=[name(g[0]) for g in GROUPS])
def test_gradients_of_heads_in_groups(case, groups, cut, sinks_cut, half):
    dtype, B, H, Hkv, Nq, Nk, d, window, sinks = case
    form = plan(*case[1:])
    heads, at = [], 0
    while at < B * Hkv:
        heads.append(min(form["group"], B * Hkv - at))
        at += heads[-1]
    assert heads == groups and (form["parts"] > 1) == cut and (sinks_cut is None or (form["sink_parts"] > 1) == sinks_cut)
    q, k, v = inputs(dtype, B, H, Hkv, Nq, Nk, d)
    do = normal((B, H, Nq, d), dtype, 4)
    kind = dtype if half else F32
    o, lse = fa2.forward_window(q, k, v, window, sinks, out_dtype=kind)
    grads = fa2.backward_window(q, k, v, o, lse, do, window, sinks, grad_dtype=kind)
    ref, bounds = backward(q, k, v, do, seen(Nq, Nk, window, sinks), 1.0 / math.sqrt(d), EPS[kind] if half else 0.0,
                           EPS[kind])
    for which, g, r, b in zip(("dQ", "dK", "dV"), grads, ref, bounds):
        assert g.dtype is kind
        close(g, r, b, which)
    again = fa2.backward_window(q, k, v, o, lse, do, window, sinks, grad_dtype=kind)
    assert torch.equal(again[1], grads[1]) and torch.equal(again[2], grads[2])

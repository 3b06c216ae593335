"""Sizes that the C interface's ints do not hold are refused, not cut to their low bits."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild

BF, HF, I32, F64 = torch.bfloat16, torch.float16, torch.int32, torch.float64
MORE = 1 << 32


class OnDevice:
    """What the Python layer looks at of a CUDA tensor, without a device or its memory."""

    is_cuda = True

    def __init__(self, *shape, dtype=BF):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", 0)
        strides = [1]
        for n in reversed(shape[1:]):
            strides.insert(0, strides[0] * max(n, 1))
        self.strides = tuple(strides)

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 4096

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True


def i32(*shape):
    return OnDevice(*shape, dtype=I32)


def cache(P=4, H=2, S=16, d=64, B=2, M=3):
    pages = OnDevice(P, H, S, d)
    return pages, pages, i32(B, M), i32(B)


FREQ = OnDevice(1, dtype=F64)

CALLS = {
    "forward: pages": lambda: fa2.forward_paged(OnDevice(2, 4, 64), *cache(P=MORE + 4)),
    "forward: slots of a page": lambda: fa2.forward_paged(OnDevice(2, 4, 64), *cache(S=MORE + 16)),
    "forward: columns of the table": lambda: fa2.forward_paged(OnDevice(2, 4, 64), *cache(M=MORE + 3)),
    "forward: sequences": lambda: fa2.forward_paged(OnDevice(2, 4, 64), *cache(B=MORE + 2), cu_q=i32(MORE + 3)),
    "forward: tokens": lambda: fa2.forward_paged(OnDevice(MORE + 2, 4, 64), *cache(), cu_q=i32(3)),
    "forward: heads": lambda: fa2.forward_paged(OnDevice(2, MORE + 4, 64), *cache()),
    "append: tokens": lambda: fa2.append_paged(OnDevice(MORE + 2, 2, 64), OnDevice(MORE + 2, 2, 64), *cache(),
                                               cu_q=i32(3)),
    "append: heads": lambda: fa2.append_paged(OnDevice(2, 2, 64), OnDevice(2, 2, 64), *cache(),
                                              q=OnDevice(2, MORE + 4, 64)),
    "rope: tokens": lambda: fa2.rope(OnDevice(1, 1, MORE + 5, 2, dtype=HF), i32(MORE + 5), FREQ),
    "rope: packed tokens": lambda: fa2.rope(OnDevice(MORE + 5, 1, 2, dtype=HF), i32(MORE + 5), FREQ),
    "rope: heads": lambda: fa2.rope_backward(OnDevice(1, MORE + 1, 5, 2, dtype=HF), i32(5), FREQ),
    "rope: batches": lambda: fa2.rope(OnDevice(MORE + 1, 1, 5, 2, dtype=HF), i32(5), FREQ),
    "rope: columns": lambda: fa2.rope(OnDevice(1, 1, 5, MORE + 2, dtype=HF), i32(5), FREQ),
    "reserve: slots of a page": lambda: fa2.pages_reserve(i32(2, 3), i32(2), i32(4), i32(2), MORE + 16),
    "reserve: pages": lambda: fa2.pages_reserve(i32(2, 3), i32(2), i32(MORE + 4), i32(2), 16),
    "reserve: sequences": lambda: fa2.pages_reserve(i32(MORE + 2, 3), i32(MORE + 2), i32(4), i32(MORE + 2), 16),
    "free: list": lambda: fa2.pages_free(i32(2, 3), i32(2), i32(4), i32(MORE + 1)),
    "compact: pages": lambda: fa2.pages_compact(i32(2, 3), i32(2), i32(MORE + 4), [OnDevice(MORE + 4, 2, 16, 64)]),
    "copy: pages": lambda: fa2.pages_copy([OnDevice(MORE + 4, 2, 16, 64)], i32(1), i32(1)),
    "copy: list": lambda: fa2.pages_copy([OnDevice(4, 2, 16, 64)], i32(MORE + 1), i32(MORE + 1)),
}


@pytest.mark.parametrize("call", CALLS)
def test_refused(call, monkeypatch):
    from contextlib import nullcontext

    from exact_attention_17_gb300 import paged

    libbuild.build()
    # past the checks: neither a device nor its memory is needed to see what would be called
    monkeypatch.setattr(paged, "_Call", lambda device, stream: nullcontext(0))
    with pytest.raises(ValueError, match="32-bit"):
        CALLS[call]()


@pytest.mark.gpu
def test_refused_on_the_device():
    libbuild.build()
    n = MORE + 5
    x = torch.ones((1, 1, 1, 2), dtype=HF, device="cuda").expand(1, 1, n, 2)
    freq = fa2.rope_inv_freq(2, device="cuda")
    pos = torch.zeros(1, dtype=I32, device="cuda").expand(n)
    held = torch.cuda.memory_allocated()
    with pytest.raises(ValueError, match="32-bit"):     # (before the positions are looked at, which are not dense)
        fa2.rope(x, pos, freq)
    table, lens, refs, add = (torch.zeros(s, dtype=I32, device="cuda") for s in ((2, 3), (2,), (4,), (2,)))
    with pytest.raises(ValueError, match="32-bit"):
        fa2.pages_reserve(table, lens, refs, add, MORE + 16)
    assert torch.cuda.memory_allocated() <= held + (1 << 20)

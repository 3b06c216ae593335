"""A cache without heads is refused as an argument, on every way into the library."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild


class OnDevice:
    """What the Python layer looks at of a CUDA tensor, without a device."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16):
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


def test_the_python_way_raises_an_argument_error():
    libbuild.build()
    i32 = lambda *s: OnDevice(*s, dtype=torch.int32)  # noqa: E731
    pages = OnDevice(4, 0, 16, 64)
    with pytest.raises(ValueError, match="heads"):
        fa2.forward_paged(OnDevice(2, 4, 64), pages, pages, i32(2, 3), i32(2))


@pytest.mark.gpu
def test_the_compiled_way_raises_an_argument_error():
    libbuild.build()
    pages = torch.empty(4, 0, 16, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((2, 3), (2,)))
    for heads in (0, 4):
        q = torch.zeros(2, heads, 64, dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ValueError, match="heads"):
            fa2.forward_paged(q, pages, pages, table, lens)
    rows = torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(fa2.FA2Error) as e:
        fa2.append_paged(rows, rows, pages, pages, table, lens, q=q)
    assert e.value.status == fa2.FA2_ERR_SHAPE

"""An output that does not fit raises torch's own out-of-memory error, so that a server can free pages and go on."""
import pytest
import torch

import exact_attention_17_gb300 as fa2
from exact_attention_17_gb300 import build as libbuild

pytestmark = pytest.mark.gpu


@pytest.fixture
def little_memory():
    libbuild.build()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    room = torch.cuda.memory_reserved() + (1 << 31)                     # 2 GB more, kept by torch's allocator
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    yield
    torch.cuda.set_per_process_memory_fraction(1.0)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("stream", [None, "given"])
def test_rope(little_memory, stream):
    x = torch.ones((1, 1, 1, 1024), device="cuda").expand(1024, 1024, 4, 1024)     # read from 4 KB, 16 GB as an output
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    freq = fa2.rope_inv_freq(1024, device="cuda")
    on = None if stream is None else torch.cuda.Stream()
    with pytest.raises(torch.OutOfMemoryError):
        fa2.rope(x, pos, freq, stream=on)
    small = fa2.rope(x[:1, :1], pos, freq, stream=on)                               # and the next call goes through
    torch.cuda.synchronize()
    assert torch.equal(small, x[:1, :1])

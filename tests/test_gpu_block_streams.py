"""The helpers that allocate, on other streams than the current one: what they
make belongs to the stream that writes it."""

import pytest
import torch

from sparse_moe_layer_03_amd import block as K
from tests.block_util import quantise_ref, say

pytestmark = pytest.mark.gpu


def owner(t):
    """The stream that torch's allocator keeps the tensor's memory for."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment holds it")


@pytest.mark.parametrize("kind", ["stream", "handle", "default", "current"])
def test_codes_belong_to_the_stream_that_writes_them(kind):
    say(f"[quantize_rows] {kind}")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    x = torch.randn((6, 50, 136), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    wq, ws = quantise_ref(x.view(300, 136))
    torch.cuda.synchronize()
    arg, handle = {"stream": (side, side.cuda_stream), "handle": (side.cuda_stream, side.cuda_stream), "default": (0, 0),
                   "current": (None, other.cuda_stream)}[kind]
    with torch.cuda.stream(other):
        q, scale = K.quantize_rows(x, stream=arg)
        e = K.I8Experts(x, x, x, stream=arg)
        assert torch.cuda.current_stream() == other
    torch.cuda.synchronize()
    made = [q, scale] + [getattr(e, f"{p}_{n}") for p in "ws" for n in ("gate", "up", "down")]
    assert [owner(t) for t in made] == [handle] * 8
    for codes, s in ((q, scale), (e.w_gate, e.s_gate), (e.w_up, e.s_up), (e.w_down, e.s_down)):
        assert torch.equal(codes.view(300, 136).double(), wq) and torch.equal(s.view(300), ws)

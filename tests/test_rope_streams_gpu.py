"""A Rope let go right after a call on another stream than its own: its
frequencies' memory must not go to other tensors before that stream has read them."""
import types

import pytest
import torch

import sparse_int4_gemm_amd as slim
from sparse_int4_gemm_amd import _lib


class Frequencies:
    device = torch.device("cuda", 0)

    def __init__(self):
        self.used_on = []

    def record_stream(self, stream):
        self.used_on.append(stream)


def test_calls_on_other_streams_are_recorded():
    own, other = types.SimpleNamespace(cuda_stream=16), types.SimpleNamespace(cuda_stream=32)
    rope = types.SimpleNamespace(freqs=Frequencies(), made_on=16, params=object())
    assert _lib._rotation(None, Frequencies.device, 16, own) is None
    assert _lib._rotation(rope, Frequencies.device, 16, own) is rope.params and rope.freqs.used_on == []
    assert _lib._rotation(rope, Frequencies.device, 32, other) is rope.params and rope.freqs.used_on == [other]


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["argument", "current"])
@pytest.mark.parametrize("call", ["rope", "append_rope", "append_q4"])
def test_its_memory_is_not_handed_out_while_a_call_waits(call, how):
    """The side stream is held up for some 50 ms; as many tensors of the frequencies' size as there may be blocks are
    taken meanwhile.  (They are not written to.)"""
    side = torch.cuda.Stream()
    x = torch.randn(3, 2, 64, device="cuda").half()
    at = torch.tensor([5, 9, 16], dtype=torch.int32, device="cuda")
    table = torch.arange(3, dtype=torch.int32, device="cuda")[:, None].contiguous()
    pools = [torch.zeros((3, 2, 16, 64), device="cuda").half() if call == "append_rope" else
             torch.zeros((3, 2, 16, 34), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty_like(x)
    want = slim.rope(x, at - int(call != "rope"), slim.Rope(64, base=777.0))
    torch.cuda.synchronize()
    rope = slim.Rope(64, base=777.0)
    place = rope.freqs.data_ptr()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    kw = {"stream": side} if how == "argument" else {}
    with torch.cuda.stream(side if how == "current" else None):
        if call == "rope":
            slim.rope(x, at, rope, out=out, **kw)
        elif call == "append_rope":
            slim.kv_append_rope(x, x, *pools, table, at, rope, q=x, q_out=out, **kw)
        else:
            slim.kv_append_q4(x, x, *pools, table, at, rope=rope, q=x, q_out=out, **kw)
    del rope
    taken = [torch.empty(32, dtype=torch.float64, device="cuda") for _ in range(100)]
    busy = not side.query()
    assert busy and place not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()
    assert torch.equal(out, want)

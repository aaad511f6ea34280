"""Calls over a 4-bit cache that share something: one workspace under several
captured graphs, pages of two sequences, the card under two streams."""
import numpy as np
import pytest

from attention_helpers import check
from q4_helpers import q4_case
from test_attention_q4_gpu import env, run  # noqa: F401

pytestmark = pytest.mark.gpu

CALLS = [([9000, 40], None), ([9000, 300], [2, 5]), ([9000, 70], [90, 60]), ([6], [6])]     # split, split few, split many, one block


def test_graphs_that_share_a_workspace(env):
    torch, slim = env
    ws = slim.workspace_attention(1, 1, 4, 2, 128)
    cs, outs, want, graphs = [], [], [], []
    for i, (lens, new) in enumerate(CALLS):
        c = q4_case(torch, 80 + i, "bf16", lens, 4, 2, 128, 64, new=new)
        want.append(run(env, c, ws=ws).clone())
        check(c, want[-1])
        cs.append(c)
        outs.append(torch.empty_like(c["q"]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            args = (c["q"], c["k4"], c["v4"], c["d_table"], c["d_lens"])
            if new is None:
                slim.attention_decode_q4(*args, scale=c["scale"], ws=ws, out=outs[-1])
            else:
                slim.attention_prefill_q4(*args, c["d_starts"], scale=c["scale"], ws=ws, out=outs[-1])
    for turn in range(3):
        ws.fill_(0xFF if ws.dtype is torch.uint8 else -1)
        for o in outs:
            o.fill_(77.0)
        for i in np.random.default_rng(turn).permutation(len(cs)):
            graphs[i].replay()
            if turn == 1:                                         # eager work between the replays
                run(env, cs[i - 1], ws=ws)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("new", [None, [3, 3, 1], [80, 80, 60]])
def test_sequences_that_share_pages(env, new):
    torch, slim = env
    c = q4_case(torch, 90, "fp16", [200, 200, 130], 4, 2, 96, 16, new=new)
    c["table"][1] = c["table"][0]
    c["table"][2] = c["table"][0]
    c["table"][2, 5] = c["table"][0, 1]                           # one page twice in a sequence
    c["d_table"].copy_(torch.from_numpy(c["table"]))
    check(c, run(env, c))


def test_two_streams_at_once(env):
    torch, slim = env
    streams = [torch.cuda.Stream() for _ in range(2)]
    cs = [q4_case(torch, 95 + i, "fp16", lens, 8, 2, 64, 32, new=new) for i, (lens, new) in enumerate(CALLS[:2])]
    want = [run(env, c).clone() for c in cs]
    ws = [slim.workspace_attention(8, 2, 8, 2, 64) for _ in cs]
    outs = [[torch.empty_like(c["q"]) for _ in range(20)] for c in cs]
    torch.cuda.synchronize()
    for turn in range(20):
        for i, c in enumerate(cs):
            args = (c["q"], c["k4"], c["v4"], c["d_table"], c["d_lens"])
            kw = dict(scale=c["scale"], ws=ws[i], out=outs[i][turn], stream=streams[i])
            if c["starts"] is None:
                slim.attention_decode_q4(*args, **kw)
            else:
                slim.attention_prefill_q4(*args, c["d_starts"], **kw)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in outs[i])

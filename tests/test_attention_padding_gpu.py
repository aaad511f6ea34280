"""Prompt attention of a padded batch whose keys are split over workgroups:
rows that belong to no sequence, before starts[0] and from starts[seqs] on, keep
what they hold, whatever the workspace held before the call."""
import numpy as np
import pytest

from attention_helpers import bound, case, host, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


def padded(env, c, first, rows, junk, **kw):
    """Output and lse of the case's tokens put at row `first` of `rows`."""
    torch, slim = env
    tokens, heads, dim = c["q"].shape
    q = torch.randn(rows, heads, dim, device="cuda").to(c["q"].dtype)
    q[first:first + tokens] = c["q"]
    out = torch.full_like(q, 77.0)
    lse = torch.full((rows, heads), 77.0, device="cuda")
    ws = slim.workspace_attention(rows, len(c["lens"]), heads, c["k"].shape[1], dim)
    ws.view(torch.float32).fill_(junk)
    slim.attention_prefill(q, c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"] + first, scale=c["scale"], ws=ws,
                           out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("junk", [3.0, float("nan"), -1.0])
@pytest.mark.parametrize("first,rows", [(0, 64), (5, 64), (5, 13), (9, 256)])
@pytest.mark.parametrize("dtype,dim", [("fp16", 128), ("bf16", 64)])
def test_rows_of_no_sequence_are_left_alone(env, dtype, dim, first, rows, junk):
    c = case(env[0], 91, dtype, [6000], 8, 2, dim, 64, new=[8])
    out, lse = padded(env, c, first, rows, junk)
    mine = slice(first, first + 8)
    want, want_lse, mass = reference(c)
    over = np.abs(host(out[mine]) - want) - bound(c, want, mass)
    assert over.max() <= 0, over.max()
    assert np.abs(host(lse[mine]) - want_lse).max() <= 2.0 ** -12 * (1 + np.abs(want_lse).max())
    for x in (out, lse):
        assert (x[:first] == 77).all() and (x[first + 8:] == 77).all()


def test_several_sequences_some_without_tokens(env):
    c = case(env[0], 92, "bf16", [4000, 50, 3000, 9], 4, 4, 64, 32, new=[5, 0, 12, 0])
    out, lse = padded(env, c, 3, 40, float("nan"))
    want, _, mass = reference(c)
    assert (np.abs(host(out[3:20]) - want) - bound(c, want, mass)).max() <= 0
    for x in (out, lse):
        assert (x[:3] == 77).all() and (x[20:] == 77).all()


def test_captured_padded_batch(env):
    """One captured call of 64 rows serves batches of any number of them."""
    torch, slim = env
    c = case(torch, 93, "fp16", [5000], 8, 2, 128, 64, new=[30])
    q, out = torch.randn(64, 8, 128, device="cuda").half(), torch.empty(64, 8, 128, device="cuda").half()
    q[:30] = c["q"]
    starts = c["d_starts"].clone()
    ws = slim.workspace_attention(64, 1, 8, 2, 128)
    call = lambda: slim.attention_prefill(q, c["k"], c["v"], c["d_table"], c["d_lens"], starts, scale=c["scale"], ws=ws, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (30, 1, 17, 30, 4):
        starts[1] = n
        out.fill_(77.0)
        graph.replay()
        got = out.clone()
        out.fill_(77.0)
        call()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and (got[n:] == 77).all()
        part = dict(c, q=q[:n], starts=np.asarray([0, n], dtype=np.int32))
        want, _, mass = reference(part)
        assert (np.abs(host(got[:n]) - want) - bound(c, want, mass)).max() <= 0

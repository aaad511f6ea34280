"""New tokens of which only some rows are given: starts that begin before row 0
or end past the last one.  The rows that exist have the positions that lens and
starts give them, in prompt attention as in kv_append."""
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


# Short (unsplit) and behind a long prefix (split).
CASES = [([300, 200], [90, 70]), ([150, 400], [150, 133]), ([5000, 4100], [20, 17])]


@pytest.mark.parametrize("lens,new", CASES)
@pytest.mark.parametrize("heads,kv_heads,dim,dtype", [(4, 1, 128, "fp16"), (2, 2, 64, "bf16")])
@pytest.mark.parametrize("skip,cut", [(0, 5), (7, 0), (13, 16), (1, 0), (0, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_rows_of_a_part_of_the_tokens(env, lens, new, heads, kv_heads, dim, dtype, skip, cut, window, sinks):
    torch, slim = env
    c = case(torch, 94, dtype, lens, heads, kv_heads, dim, 16, new=new)
    rows = slice(skip, sum(new) - cut)
    q = c["q"][rows]
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    slim.attention_prefill(q, c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"] - skip, window=window, sinks=sinks,
                           scale=c["scale"], out=out, lse=lse)
    torch.cuda.synchronize()
    want, want_lse, mass = (x[rows] for x in reference(c, window, sinks))
    over = np.abs(host(out) - want) - bound(c, want, mass)
    assert over.max() <= 0, over.max()
    assert np.abs(host(lse) - want_lse).max() <= 2.0 ** -12 * (1 + np.abs(want_lse).max())


@pytest.mark.parametrize("starts", [[-2 ** 31, -5, 20], [-2 ** 31, 20, 2 ** 31 - 1], [0, 10, 2 ** 31 - 1], [-300, 40, 500]])
def test_far_starts(env, starts):
    """As many tokens before row 0 or past the last as an int32 holds."""
    torch, slim = env
    c = case(torch, 95, "fp16", [300, 250], 2, 1, 64, 16, new=[30, 30])
    q = c["q"]
    out = torch.full_like(q, 77.0)
    slim.attention_prefill(q, c["k"], c["v"], c["d_table"], c["d_lens"], torch.tensor(starts, dtype=torch.int32, device="cuda"),
                           scale=c["scale"], out=out)
    torch.cuda.synchronize()
    got = host(out)
    for t in range(60):
        b = next((b for b in range(2) if starts[b] <= t < starts[b + 1]), None)
        if b is None:
            assert (got[t] == 77).all()
            continue
        p = int(c["lens"][b]) - (starts[b + 1] - t)                  # one row at its position
        one = dict(c, q=q[t:t + 1], table=c["table"][b:b + 1], lens=np.asarray([max(p + 1, 0)]), starts=np.asarray([0, 1]))
        want, _, mass = reference(one)
        assert (np.abs(got[t] - want[0]) - bound(c, want[0], mass[0])).max() <= 0, t


def test_append_and_attention_agree_on_positions(env):
    """Appending a part of the tokens and attending with it sees its own keys last."""
    torch, slim = env
    c = case(torch, 96, "fp16", [100], 2, 2, 64, 16, new=[40])
    full = torch.randn(40, 2, 64, device="cuda").half()
    slim.kv_append(full, full, c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"])
    k0, v0 = c["k"].clone(), c["v"].clone()
    for skip, cut in ((6, 0), (0, 9), (3, 4)):
        rows = slice(skip, 40 - cut)
        c["k"][:], c["v"][:] = k0, v0
        for j in range(60 + skip, 100 - cut):
            c["k"][int(c["table"][0, j // 16]), :, j % 16] = 0
            c["v"][int(c["table"][0, j // 16]), :, j % 16] = 0
        slim.kv_append(full[rows], full[rows], c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"] - skip)
        torch.cuda.synchronize()
        assert torch.equal(c["k"], k0) and torch.equal(c["v"], v0)

"""The orders in which attention's workgroups take their work, and where the
wave groups change: many uneven sequences (longest first), whole prompts on
both sides of the rules, second rounds of workgroups.  Against the fp64 oracle
with the bound of the attention tests; the order changes no result."""
import numpy as np
import pytest

from attention_helpers import case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


def run(env, c, window=0, sinks=0, **kw):
    torch, slim = env
    out = torch.full_like(c["q"], 77.0)
    lse = torch.full(c["q"].shape[:2], 77.0, device="cuda")
    kw = dict(window=window, sinks=sinks, scale=c["scale"], out=out, lse=lse, **kw)
    args = (c["q"], c["k"], c["v"], c["d_table"], c["d_lens"])
    if c["starts"] is None:
        slim.attention_decode(*args, **kw)
    else:
        slim.attention_prefill(*args, c["d_starts"], **kw)
    torch.cuda.synchronize()
    return out, lse


def uneven(seqs, most, seed):
    lens = np.random.default_rng(seed).integers(0, most + 1, seqs)
    lens[[0, 1, 2, seqs // 2, -2, -1]] = [most, 0, 1, most, 16, most]
    return [int(n) for n in lens]


@pytest.mark.parametrize("seqs,heads,kv_heads,dim", [(65, 16, 8, 64), (130, 8, 8, 128), (64, 40, 10, 96), (257, 4, 2, 256),
                                                     (33, 40, 20, 64), (600, 17, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (520, 9)])
def test_uneven_batches_of_single_tokens(env, seqs, heads, kv_heads, dim, window, sinks):
    c = case(env[0], 81, "bf16", uneven(seqs, 700, seqs), heads, kv_heads, dim, 32)
    y, lse = run(env, c, window, sinks)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("max_len", [511, 512, 600, 5000, 1 << 30])
def test_the_expected_length_changes_no_result(env, max_len):
    torch, _ = env
    c = case(torch, 82, "fp16", uneven(150, 640, 82), 8, 4, 64, 16)
    y, lse = run(env, c, max_len=max_len)
    check(c, y, lse)
    y1, lse1 = run(env, c, max_len=16)            # in the batch's own order
    assert torch.equal(y, y1) and torch.equal(lse, lse1)


def test_equal_and_out_of_range_lengths(env):
    torch, _ = env
    c = case(torch, 83, "fp16", [512] * 140, 4, 4, 64, 16)
    y, lse = run(env, c)
    check(c, y, lse)
    c["lens"] = c["lens"].copy()
    c["lens"][[3, 70, 139]] = [-5, 1 << 30, np.iinfo(np.int32).max]
    c["d_lens"].copy_(torch.from_numpy(c["lens"]))
    c["lens"][139] = 1 << 30                      # lengths are taken to be at most 2^30
    y, lse = run(env, c)
    check(c, y, lse)


def test_replays_follow_the_lengths(env):
    """A captured call orders the sequences by the lengths of each replay."""
    torch, slim = env
    c = case(torch, 84, "bf16", [640] * 140, 4, 4, 64, 32)
    ws = slim.workspace_attention(140, 140, 4, 4, 64)
    out = torch.empty_like(c["q"])
    call = lambda o: slim.attention_decode(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], scale=c["scale"], ws=ws, out=o)
    call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for seed in range(4):
        c["lens"] = np.asarray(uneven(140, 640, seed), dtype=np.int32)
        c["d_lens"].copy_(torch.from_numpy(c["lens"]))
        out.fill_(77.0)
        graph.replay()
        eager = torch.empty_like(out)
        call(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        check(c, out)


@pytest.mark.parametrize("dtype,dim,heads,kv_heads", [("fp16", 64, 96, 96), ("bf16", 96, 96, 96), ("bf16", 128, 128, 32),
                                                      ("fp16", 256, 96, 96)])
@pytest.mark.parametrize("new,pre", [(390, 0), (390, 90), (390, 300)])
def test_whole_prompts_and_chunks_past_one_round(env, dtype, dim, heads, kv_heads, new, pre):
    """More row blocks than 256: in two wave groups for whole prompts, in one behind a prefix."""
    c = case(env[0], 85, dtype, [new + pre], heads, kv_heads, dim, 64, new=[new])
    y, lse = run(env, c)
    check(c, y, lse)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("window,sinks", [(100, 0), (150, 70), (590, 5), (0, 0)])
def test_prompt_past_two_rounds(env, dim, window, sinks):
    c = case(env[0], 86, "bf16", [601], 112, 112, dim, 128, new=[601])
    y, lse = run(env, c, window, sinks)
    check(c, y, lse, window, sinks)

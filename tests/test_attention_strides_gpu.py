"""The widest rows and the longest row strides that the attention and cache
calls take."""
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


def run(env, c, **kw):
    torch, slim = env
    args = (c["q"], c["k"], c["v"], c["d_table"], c["d_lens"])
    if c["starts"] is None:
        return slim.attention_decode(*args, scale=c["scale"], **kw)
    return slim.attention_prefill(*args, c["d_starts"], scale=c["scale"], **kw)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(1024, 64, 128), (1024, 1024, 64), (512, 8, 256)])
def test_rows_of_many_heads(env, form, heads, kv_heads, dim):
    c = case(env[0], 111, "bf16", [5, 40], heads, kv_heads, dim, 16, new=None if form == "decode" else [2, 3])
    check(c, run(env, c))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_rows_far_apart(env, form):
    torch, slim = env
    new = None if form == "decode" else [100, 30]
    c = case(torch, 112, "fp16", [120, 35] if new else [1 + i for i in range(130)], 4, 2, 64, 16, new=new)
    want = run(env, c)
    tokens, stride = c["q"].shape[0], 1 << 22
    far_q, far_o = (torch.empty(tokens * stride, dtype=torch.float16, device="cuda").as_strided((tokens, 4, 64), (stride, 64, 1))
                    for _ in range(2))
    far_q.copy_(c["q"])
    assert torch.equal(run(env, dict(c, q=far_q), out=far_o), want)
    pools = [(c["k"].clone(), c["v"].clone()) for _ in range(2)]
    slim.kv_append(c["q"][:, :2], c["q"][:, 2:], *pools[0], c["d_table"], c["d_lens"], c["d_starts"])
    slim.kv_append(far_q[:, :2], far_q[:, 2:], *pools[1], c["d_table"], c["d_lens"], c["d_starts"])
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    with pytest.raises(slim.SlimError):
        far = torch.empty(2 * stride + 1024, dtype=torch.float16, device="cuda").as_strided((2, 4, 64), (stride + 8, 64, 1))
        slim.attention_decode(far, c["k"], c["v"], c["d_table"][:2].contiguous(), c["d_lens"][:2].contiguous())

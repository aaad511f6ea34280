"""How many bits the softmax weights keep: in single-token attention those of
fp32 (each enters the product as a high and a low half), in both forms also
weights far below the largest, of which a long cache has many."""
import numpy as np
import pytest

from attention_helpers import UNIT, case, host, reference

TYPES = {"fp16": "float16", "bf16": "bfloat16"}


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


def tight(dtype, out, mass):
    """With u the type's unit roundoff: |o| u for the output's rounding; a
    weight whose low half is rounded is off by u^2 of itself; exact scores
    leave 2^-20 for the exponentials (a product and an exponential of 2^-23 each)
    and sums of 64 terms in fp32.  A tenth for second-order terms."""
    u = UNIT[dtype]
    return 1.1 * (np.abs(out) * u + mass * (u * u + 2.0 ** -20)) + 2.0 ** -24


def exact_scores(torch, dtype, device):
    """32 sequences of 64 keys whose scores are multiples of 2^-8 in (-1, 0], in one element of the keys."""
    rng = np.random.default_rng(101)
    td = getattr(torch, TYPES[dtype])
    k = np.zeros((32, 1, 64, 64), dtype=np.float32)
    k[..., 5] = -rng.integers(0, 256, (32, 1, 64)) / 256.0
    q = np.zeros((32, 2, 64), dtype=np.float32)
    q[:, 0, 5], q[:, 1, 5] = 1.0, 2.0
    v = rng.standard_normal((32, 1, 64, 64), dtype=np.float32)
    q, k, v = (torch.from_numpy(x).to(td).to(device) for x in (q, k, v))
    assert np.array_equal(host(k[..., 5]), host(k[..., 5].float()))
    return dict(q=q, k=k, v=v, table=np.arange(32, dtype=np.int32)[:, None], lens=np.full(32, 64, dtype=np.int32),
                starts=None, scale=1.0, dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weights_of_one_rounding_are_outside_the_bound(dtype):
    """(The bound below tells the two apart.)"""
    torch = pytest.importorskip("torch")
    c = exact_scores(torch, dtype, "cpu")
    out, _, mass = reference(c)
    k, q, v = host(c["k"])[:, 0], host(c["q"]), host(c["v"])[:, 0]
    w = np.exp(q @ k.transpose(0, 2, 1) - (q @ k.transpose(0, 2, 1)).max(-1, keepdims=True))
    once = host(torch.from_numpy(w).to(getattr(torch, TYPES[dtype])))
    assert (np.abs(w @ v / w.sum(-1, keepdims=True) - out) <= tight(dtype, out, mass)).all()
    over = np.abs(once @ v / w.sum(-1, keepdims=True) - out) - tight(dtype, out, mass)
    assert (over > 0).mean() > 0.02


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_single_token_weights_keep_the_bits_of_fp32(env, dtype):
    torch, slim = env
    c = exact_scores(torch, dtype, "cuda")
    got = host(slim.attention_decode(c["q"], c["k"], c["v"], torch.from_numpy(c["table"]).cuda(),
                                     torch.from_numpy(c["lens"]).cuda(), scale=1.0))
    out, _, mass = reference(c)
    over = np.abs(got - out) - tight(dtype, out, mass)
    assert over.max() <= 0, over.max()


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", [0, None], ids=["whole", "split"])
@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bits", [14, 20, 25.5, 28])
def test_many_small_weights_beside_a_large_first_one(env, form, dtype, bits, max_len):
    """Key 0 has score bits * ln 2, 2^19 - 1 others 0, and all values are 1: the
    output is 1, whatever share the others have (2^19 2^-bits: 1% at 25.5, where
    an fp16 weight relative to the largest would be 0).  Beside the output's rounding and
    (prompts) one of the weights, it may be off by 2^-24 for each addition one after another
    to the sum and to the output, of 32 keys a wave and step (of four waves, two
    products each, or of two groups' 16 keys a product), and by half of fp16's smallest
    number, 2^-25, behind weights of at least 2^7 for the largest, per key."""
    torch, slim = env
    n = 1 << 19
    new = None if form == "decode" else [3]
    c = case(torch, 102, dtype, [n], 2, 1, 64, 1024, new=new)
    c["k"].zero_()
    c["v"].fill_(1.0)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    high = torch.tensor(bits * np.log(2.0)).to(c["k"].dtype)
    c["k"][int(c["table"][0, 0]), 0, 0, 0] = high
    args = (c["q"], c["k"], c["v"], c["d_table"], c["d_lens"])
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    kw = dict(scale=1.0, lse=lse, max_len=max_len)
    got = slim.attention_decode(*args, **kw) if new is None else slim.attention_prefill(*args, c["d_starts"], **kw)
    u = UNIT[dtype]
    sums = n // 128 if form == "decode" else n // 64
    off = (u + u * u if form == "decode" else 2 * u) + (sums + 2 * sums) * 2.0 ** -24 + n * 2.0 ** -32
    assert np.abs(host(got) - 1.0).max() <= off, np.abs(host(got) - 1.0).max()
    seen = np.asarray([n]) if new is None else np.arange(n - 2, n + 1)
    want = np.log(np.exp(float(high)) + seen - 1)
    assert np.abs(host(lse) - want[:, None]).max() <= sums * 2.0 ** -24 + 2.0 ** -15 * (1 + want.max())

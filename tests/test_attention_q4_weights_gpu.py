"""How many bits the softmax weights keep over a cache of 4 bits: those of fp32,
for single tokens and for batches of few rows (a high and a low half of each enter
the products)."""
import numpy as np
import pytest

from attention_helpers import host, reference
from oracle import q4_ref
from test_attention_weights_gpu import TYPES, tight


def exact_scores(torch, dtype, dim, device):
    """32 sequences of 64 keys whose scores are multiples of 2^-8 in (-1, 0], in one element of each of the keys'
    first two groups of 32, whose scales are 2^-3 and 2^-7; one new token each."""
    rng = np.random.default_rng(103)
    code = np.zeros((32, 1, 64, dim), dtype=np.uint8)
    scale = np.full((32, 1, 64, dim // 32), 127, dtype=np.uint8)
    code[..., 5], code[..., 37] = 8 + rng.integers(0, 8, (2, 32, 1, 64))
    scale[..., 0], scale[..., 1] = 127 - 3, 127 - 7
    v_code = rng.integers(0, 16, code.shape, dtype=np.uint8)
    v_scale = np.full_like(scale, 127)
    q = np.zeros((32, 2, dim), dtype=np.float32)
    q[:, 0, 5] = q[:, 0, 37] = 1.0
    q[:, 1, 5] = q[:, 1, 37] = 2.0
    td = getattr(torch, TYPES[dtype])
    k, v = q4_ref.decode(code, scale), q4_ref.decode(v_code, v_scale)
    return dict(q=torch.from_numpy(q).to(td).to(device), k=torch.from_numpy(k).to(td), v=torch.from_numpy(v).to(td),
                k4=torch.from_numpy(q4_ref.pack(code, scale)).to(device),
                v4=torch.from_numpy(q4_ref.pack(v_code, v_scale)).to(device),
                table=np.arange(32, dtype=np.int32)[:, None], lens=np.full(32, 64, dtype=np.int32),
                starts=None, scale=1.0, dtype=dtype)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weights_of_one_rounding_are_outside_the_bound(dtype, dim):
    """(The bound below tells the two apart.)"""
    torch = pytest.importorskip("torch")
    c = exact_scores(torch, dtype, dim, "cpu")
    out, _, mass = reference(c)
    k, q, v = host(c["k"])[:, 0], host(c["q"]), host(c["v"])[:, 0]
    s = q @ k.transpose(0, 2, 1)
    assert (s == np.round(s * 256) / 256).all() and s.min() >= -2 and len(np.unique(s[:, 0])) > 30
    w = np.exp(s - s.max(-1, keepdims=True))
    once = host(torch.from_numpy(w).to(getattr(torch, TYPES[dtype])))
    assert (np.abs(w @ v / w.sum(-1, keepdims=True) - out) <= tight(dtype, out, mass)).all()
    over = np.abs(once @ v / w.sum(-1, keepdims=True) - out) - tight(dtype, out, mass)
    assert (over > 0).mean() > 0.02


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["single", "few rows"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weights_keep_the_bits_of_fp32(dtype, dim, form):
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    c = exact_scores(torch, dtype, dim, "cuda")
    args = (c["q"], c["k4"], c["v4"], torch.from_numpy(c["table"]).cuda(), torch.from_numpy(c["lens"]).cuda())
    if form == "single":
        got = slim.attention_decode_q4(*args, scale=1.0)
    else:
        got = slim.attention_prefill_q4(*args, torch.arange(33, device="cuda", dtype=torch.int32), scale=1.0)
    out, _, mass = reference(c)
    over = np.abs(host(got) - out) - tight(dtype, out, mass)
    assert over.max() <= 0, over.max()

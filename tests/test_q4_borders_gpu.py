"""Which numbers choose a turned key's code: those of the rotation in fp64, its
magnitude too, held in fp32.  Keys whose turned elements lie next to a border
between two codes, so near that a turn in fp32, or a magnitude rounded to fp32,
takes another code for many of them."""
import math

import numpy as np
import pytest

from attention_helpers import host
from oracle import q4_ref, rope_ref

MAGNITUDES = [1.0, 0.1 * math.log(40.0) + 1.0, 1.0 + 2.0 ** -24, 0.7]       # none, yarn's at factor 40, others
BORDERS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def half(x, dtype):
    """The numbers of the type nearest x, towards zero in bf16."""
    if dtype == "fp16":
        return np.float64(np.float16(x))
    return np.float64((np.float32(x).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32))


def keys_at_borders(seed, magnitude, dtype):
    """One row of 16 heads of 128 and the frequencies of its pairs 2 i, 2 i + 1 at position 1.  The
    first pair of every 32 elements is (6, 0.4), not turned, so that the group's scale is 1 (nothing exceeds 7);
    of every other pair of head 0 the first element comes to lie 0.52 of an fp32 step above or below a border,
    or on it."""
    rng = np.random.default_rng(seed)
    x = np.zeros((1, 16, 128))
    freqs = np.zeros(64)
    x[:, :, ::32], x[:, :, 1::32] = half(6.0 / magnitude, dtype), half(0.4 / magnitude, dtype)
    for i in range(64):
        if i % 16 == 0:
            continue
        border = rng.choice(BORDERS) * rng.choice((-1.0, 1.0))
        step = float(np.spacing(np.float32(abs(border))))
        at = (border + step * rng.choice((-0.52, 0.0, 0.52))) / magnitude
        while True:
            a, b = (float(half(t, dtype)) for t in rng.uniform(-6.9, 6.9, 2) / magnitude)
            r = math.hypot(a, b)
            if abs(at) < 0.98 * r < 0.98 * 6.9 / magnitude:
                break
        # a cos t - b sin t = r cos(t + atan2(b, a))
        freqs[i] = math.acos(at / r) - math.atan2(b, a)
        x[0, 0, 2 * i:2 * i + 2] = a, b
    x[0, 1:] = x[0, 0] * rng.choice((-1.0, 1.0), (15, 1))
    return x, freqs


def turned_in_fp32(x, freqs, magnitude):
    c, s = (np.float32(magnitude * f(freqs)) for f in (np.cos, np.sin))
    a, b = np.float32(x[..., 0::2]), np.float32(x[..., 1::2])
    y = np.empty(x.shape, dtype=np.float32)
    y[..., 0::2], y[..., 1::2] = a * c - b * s, b * c + a * s
    return y


def turned(x, freqs, magnitude):
    return rope_ref.turn(x, [1], freqs, True, magnitude).astype(np.float32)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("magnitude", MAGNITUDES)
def test_other_roundings_take_other_codes(magnitude, dtype):
    """(The test below tells them apart.)"""
    shifted = single = elements = 0
    for seed in range(20):
        x, freqs = keys_at_borders(seed, magnitude, dtype)
        code, scale = q4_ref.encode(turned(x, freqs, magnitude), dtype)
        assert (scale == 127).all()
        single += (q4_ref.encode(turned_in_fp32(x, freqs, magnitude), dtype)[0] != code).sum()
        shifted += (q4_ref.encode(turned(x, freqs, float(np.float32(magnitude))), dtype)[0] != code).sum()
        elements += 16 * 60
    assert single > 0.05 * elements, single
    assert magnitude == 1.0 or shifted > 0.05 * elements, shifted


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("magnitude", MAGNITUDES)
def test_codes_are_those_of_the_rotation_in_fp64(magnitude, dtype):
    """Also of many tokens, which another form of the kernel appends."""
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    for seed in range(20):
        x, freqs = keys_at_borders(seed, magnitude, dtype)
        code, scale = q4_ref.encode(turned(x, freqs, magnitude), dtype)
        rope = slim.Rope(128, freqs=torch.from_numpy(freqs), interleaved=True, magnitude=magnitude)
        assert rope.magnitude == magnitude
        for tokens in (1, 600):
            k = torch.from_numpy(x).to(getattr(torch, {"fp16": "float16", "bf16": "bfloat16"}[dtype])).cuda()
            k = k.expand(tokens, 16, 128).contiguous()
            assert np.array_equal(host(k[:1]), x)
            pool = [torch.zeros((tokens, 16, 16, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
            table = torch.arange(tokens, device="cuda", dtype=torch.int32)[:, None].contiguous()
            slim.kv_append_q4(k, k, *pool, table, torch.full((tokens,), 2, dtype=torch.int32, device="cuda"), rope=rope)
            torch.cuda.synchronize()
            got_code, got_scale = q4_ref.unpack(pool[0].cpu().numpy())
            assert (got_code[:, :, 1] == code).all() and (got_scale[:, :, 1] == scale).all(), (seed, tokens)

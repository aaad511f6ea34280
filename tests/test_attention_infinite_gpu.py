"""Infinite and NaN values that a single-token row sees: its element is what
the formula gives, +-inf for infinities of one sign and NaN for both signs or a
NaN, whatever the weight's rounding; every other element and row is as if the
value were finite."""
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


def weights(c, b, h):
    """Softmax weights of sequence b's keys for query head h, relative to the largest."""
    n, share = int(c["lens"][b]), c["q"].shape[1] // c["k"].shape[1]
    j = np.arange(n)
    page = c["k"].shape[2]
    k = host(c["k"][c["table"][b, j // page].tolist(), h // share, (j % page).tolist()])
    s = k @ host(c["q"][b, h]) * c["scale"]
    return np.exp(s - s.max())


def decode(env, c, **kw):
    torch, slim = env
    lse = torch.full(c["q"].shape[:2], 77.0, device="cuda")
    out = slim.attention_decode(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], scale=c["scale"], lse=lse, **kw)
    torch.cuda.synchronize()
    return host(out), host(lse)


def put(c, b, j, head, element, value):
    page = c["k"].shape[2]
    c["v"][int(c["table"][b, j // page]), head, j % page, element] = value


def places(c, pick):
    """A key of each sequence: the largest weight's of some head, or one of its rank in `pick`."""
    keys = []
    for b in range(len(c["lens"])):
        order = np.argsort(-weights(c, b, b % c["q"].shape[1]))
        keys.append(int(order[min(pick[b % len(pick)], len(order) - 1)]))
    return keys


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 4, 2), (96, 2, 1), (128, 20, 1), (128, 3, 3), (256, 16, 1)])
@pytest.mark.parametrize("lens", [[90] * 40 + [1, 1, 17, 33], [6000, 5200, 4100]], ids=["whole", "split"])
def test_a_seen_infinity(env, dtype, dim, heads, kv_heads, lens):
    torch, _ = env
    c = case(torch, 97, dtype, lens, heads, kv_heads, dim, 16)
    want, want_lse, mass = reference(c)
    keys = places(c, [0, 0, 1, 2, 5, 11, 29, 60])
    share, half = heads // kv_heads, {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    low = []
    for b, j in enumerate(keys):
        head = b % kv_heads
        put(c, b, j, head, (5 * b + 3) % dim, float("inf") if b % 2 else float("-inf"))
        w = np.asarray([weights(c, b, h)[j] for h in range(head * share, (head + 1) * share)])
        low += list(w - host(torch.from_numpy(w).to(half)))
    if len(lens) > 3:                           # weights of all kinds: whole, rounded up, rounded down
        low = np.asarray(low)
        assert (low == 0).any() and (low > 0).any() and (low < 0).any()
    got, lse = decode(env, c)
    for b in range(len(lens)):
        head, e = b % kv_heads, (5 * b + 3) % dim
        mine = slice(head * share, (head + 1) * share)
        assert (got[b, mine, e] == (np.inf if b % 2 else -np.inf)).all(), (b, keys[b], got[b, mine, e])
        got[b, mine, e] = want[b, mine, e]
    over = np.abs(got - want) - bound(c, want, mass)
    assert over.max() <= 0, np.unravel_index(over.argmax(), over.shape)
    assert np.abs(lse - want_lse).max() <= 2.0 ** -12 * (1 + np.abs(want_lse).max())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("lens", [[90] * 6, [6000]], ids=["whole", "split"])
def test_infinities_of_both_signs_and_nan(env, dtype, lens):
    torch, _ = env
    c = case(torch, 98, dtype, lens, 4, 2, 128, 32)
    want, _, mass = reference(c)
    for b, n in enumerate(lens):
        put(c, b, 3, 0, 7, float("inf"))
        put(c, b, n - 2, 0, 7, float("-inf"))
        put(c, b, n // 2, 0, 8, float("nan"))
        put(c, b, 5, 0, 9, float("inf"))
        put(c, b, n - 1, 0, 9, float("inf"))
    got, _ = decode(env, c)
    assert np.isnan(got[:, :2, 7:9]).all() and np.isposinf(got[:, :2, 9]).all()
    got[:, :2, 7:10] = want[:, :2, 7:10]
    assert (np.abs(got - want) - bound(c, want, mass)).max() <= 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (700, 0)])
def test_the_window_decides_who_sees_it(env, dtype, window, sinks):
    """The same keys, infinite in every sequence, inside the window of some only."""
    torch, slim = env
    lens = [1, 2, 40, 41, 64, 100, 300, 1000, 5000]
    c = case(torch, 99, dtype, lens, 4, 1, 64, 16)
    want, _, mass = reference(c, window, sinks)
    for b, n in enumerate(lens):
        for j in (0, 39, 290, 990):
            if j < n:
                put(c, b, j, 0, j % 64, float("inf"))
    got, _ = decode(env, c, window=window, sinks=sinks)
    for b, n in enumerate(lens):
        for j in (0, 39, 290, 990):
            if j < n and (not window or j > n - 1 - window or j < sinks):
                assert np.isposinf(got[b, :, j % 64]).all(), (n, j)
                got[b, :, j % 64] = want[b, :, j % 64]
    assert (np.abs(got - want) - bound(c, want, mass)).max() <= 0


def test_the_two_forms_agree(env):
    """A row of a prompt and the same row as a single token."""
    torch, slim = env
    for dtype in ("fp16", "bf16"):
        c = case(torch, 100, dtype, [77] * 12, 4, 2, 128, 16)
        want, _, mass = reference(c)
        for b in range(12):
            put(c, b, 6 * b + 1, b % 2, b, float("inf"))
        one, _ = decode(env, c)
        starts = torch.arange(13, dtype=torch.int32, device="cuda")
        two = host(slim.attention_prefill(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], starts, scale=c["scale"]))
        assert np.array_equal(np.isposinf(one), np.isposinf(two)) and np.isposinf(one).sum() == 24
        assert not np.isnan(one).any() and not np.isnan(two).any()
        fine = np.isfinite(one)
        assert (np.abs(one[fine] - two[fine]) <= 2 * bound(c, want, mass)[fine]).all()

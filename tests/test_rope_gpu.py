"""slim_rope and slim_kv_append_rope against the fp64 oracle and against each
other: types, layouts, parts of a head, odd sizes, far and negative positions,
in place, strides, streams, graphs, and rows and places that must stay."""
import numpy as np
import pytest

from attention_helpers import UNIT, case, host
from oracle import attention_ref, rope_ref

pytestmark = pytest.mark.gpu
TYPES = {"fp16": "float16", "bf16": "bfloat16"}


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


def rows(torch, dtype, *shape, seed=1, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(getattr(torch, TYPES[dtype]))


def ints(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(got, x, positions, rope, dtype, what=""):
    """Bound: the output's own rounding (half a step, u of the value, fp16's
    subnormal step below its normal range); cos and sin rounded to fp32 and two
    products and a sum in fp32, 4 roundings of 2^-24 of |a| + |b|; and the angle, two fp64
    roundings here and one in the oracle, each 2^-53 of p * f, f at most 1."""
    f = rope.freqs.cpu().numpy()
    want = rope_ref.turn(x, positions, f, rope.interleaved, rope.magnitude)
    reach = abs(rope.magnitude) * (np.abs(x) + rope_ref.partner(x, len(f), rope.interleaved))
    p = np.abs(np.asarray(positions, dtype=np.float64))[:, None, None]
    limit = np.abs(want) * UNIT[dtype] + reach * (4 * 2.0 ** -24 + 3 * p * 2.0 ** -53) + 2.0 ** -25
    over = np.abs(got - want) - 1.01 * limit
    assert np.isfinite(got).all() and over.max(initial=-1) <= 0, f"{what}: {over.max():.3e} at {np.unravel_index(over.argmax(), over.shape)}"
    n = 2 * len(f)
    assert np.array_equal(got[..., n:], x[..., n:]), f"{what}: elements that are not turned"


# --------------------------------------------------------------------- rope
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", [
    (1, 1, 8, 8), (1, 32, 128, 128), (3, 5, 64, 16), (7, 3, 96, 24), (33, 2, 96, 96), (5, 7, 128, 40), (2, 1, 256, 256),
    (4, 3, 72, 16), (2, 2, 72, 72), (3, 1, 1024, 1024), (1, 1024, 64, 64), (600, 3, 80, 32), (513, 20, 128, 64), (700, 1, 24, 8)])
def test_rope(env, dtype, interleaved, tokens, heads, dim, rot):
    torch, slim = env
    rope = slim.Rope(rot, interleaved=interleaved)
    x = rows(torch, dtype, tokens, heads, dim)
    at = np.random.default_rng(tokens).integers(0, 5000, tokens)
    y = slim.rope(x, ints(torch, at), rope)
    torch.cuda.synchronize()
    check(host(y), host(x), at, rope, dtype)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rope_far_negative_and_scaled_positions(env, scaling):
    torch, slim = env
    rope = slim.Rope(64, scaling=scaling, factor=8.0, original_len=4096, interleaved=True)
    at = [0, 1, -1, 4095, 131072, -131072, 2 ** 30, -2 ** 30, 2 ** 31 - 1, -2 ** 31, 999999937]
    x = rows(torch, "fp16", len(at), 4, 96)
    y = slim.rope(x, ints(torch, at), rope)
    torch.cuda.synchronize()
    check(host(y), host(x), at, rope, "fp16")


def test_turning_back_is_the_inverse_and_the_gradient(env):
    torch, slim = env
    for interleaved in (False, True):
        rope = slim.Rope(96, interleaved=interleaved, magnitude=1.25)
        at = np.arange(50) * 37
        x, g = rows(torch, "bf16", 50, 3, 128), rows(torch, "bf16", 50, 3, 128, seed=2)
        back = slim.rope(g, ints(torch, -at), rope)
        torch.cuda.synchronize()
        check(host(back), host(g), -at, rope, "bf16")
        # d <g, y(x)> / dx along some directions, by differences of the (linear) formula.
        f = rope.freqs.cpu().numpy()
        want = rope_ref.turn(host(g), -at, f, interleaved, 1.25)
        rng = np.random.default_rng(3)
        for _ in range(3):
            d = rng.standard_normal(x.shape) * (np.arange(128) < 96)
            y = [rope_ref.turn(host(x) + s * d, at, f, interleaved, 1.25) for s in (0.5, -0.5)]
            assert np.isclose((host(g) * (y[0] - y[1])).sum(), (want * d).sum(), rtol=1e-9)
        once = slim.Rope(96, interleaved=interleaved)
        y = slim.rope(slim.rope(x, ints(torch, at), once), ints(torch, -at), once)
        torch.cuda.synchronize()
        # Two roundings of 2^-8 and their reach through the rotation (both elements of the pair).
        reach = np.abs(host(x)) + rope_ref.partner(host(x), 48, interleaved)
        assert (np.abs(host(y) - host(x)) <= 3 * 2.0 ** -8 * reach + 1e-30).all()


@pytest.mark.parametrize("tokens", [5, 700])
@pytest.mark.parametrize("interleaved,dim,rot", [(False, 128, 128), (True, 128, 64), (False, 96, 24), (True, 72, 16)])
def test_rope_in_place_and_strided(env, tokens, interleaved, dim, rot):
    torch, slim = env
    rope = slim.Rope(rot, interleaved=interleaved)
    at = ints(torch, np.arange(tokens) + 11)
    x = rows(torch, "fp16", tokens, 6, dim)
    want = slim.rope(x, at, rope)
    joint = rows(torch, "fp16", tokens, 11, dim, seed=5)
    joint[:, 2:8] = x
    before = joint.clone()
    wide = torch.full((tokens, 9, dim), 77.0, device="cuda", dtype=torch.float16)
    got = slim.rope(joint[:, 2:8], at, rope, out=wide[:, 1:7])
    assert torch.equal(got, want) and (wide[:, :1] == 77).all() and (wide[:, 7:] == 77).all()
    part = joint[:, 2:8]
    assert slim.rope(part, at, rope, out=part) is part
    torch.cuda.synchronize()
    assert torch.equal(part, want) and torch.equal(joint[:, :2], before[:, :2]) and torch.equal(joint[:, 8:], before[:, 8:])
    for i in range(tokens if tokens < 9 else 0):                       # one row at a time: the same bits
        assert torch.equal(slim.rope(x[i:i + 1], at[i:i + 1], rope), want[i:i + 1])


def test_rope_keeps_infinities_and_nan_in_their_pairs(env):
    torch, slim = env
    rope = slim.Rope(64)
    x = rows(torch, "fp16", 3, 2, 128)
    at = ints(torch, [4, 5, 6])
    clean = slim.rope(x, at, rope).clone()
    x[1, 1, 3], x[2, 0, 100] = float("nan"), float("inf")
    y = slim.rope(x, at, rope)
    torch.cuda.synchronize()
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, 1, 3] = hit[1, 1, 35] = hit[2, 0, 100] = True
    assert torch.equal(y[~hit], clean[~hit]) and y[1, 1, [3, 35]].isnan().all() and y[2, 0, 100] == float("inf")


def test_rope_streams_graphs_and_empty(env):
    torch, slim = env
    rope = slim.Rope(128)
    x = rows(torch, "bf16", 9, 8, 128)
    at = ints(torch, np.arange(9) * 100)
    want = slim.rope(x, at, rope)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = slim.rope(x, at, rope, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slim.rope(x, at, rope, out=out)
    for turn in range(3):
        x.copy_(rows(torch, "bf16", 9, 8, 128, seed=20 + turn))
        at.copy_(ints(torch, np.arange(9) * 7 + turn))
        out.fill_(77.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, slim.rope(x, at, rope))
    assert slim.rope(x[:0], at[:0], rope).shape == (0, 8, 128)


def test_rope_refusals_in_the_binding(env):
    torch, slim = env
    rope = slim.Rope(64)
    x, at = rows(torch, "fp16", 4, 2, 128), ints(torch, [0, 1, 2, 3])
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(positions=at.long()), dict(positions=at[:3]), dict(out=x[:3]),
                dict(out=x.bfloat16()), dict(x=x.transpose(0, 1)), dict(x=x[:, :, ::2]), dict(rope=slim.Rope(64, device="cpu")),
                dict(x=x[..., :12]), dict(rope=slim.Rope(256))):
        with pytest.raises((TypeError, ValueError, slim.SlimError)):
            slim.rope(**{**dict(x=x, positions=at, rope=rope), **bad})


# -------------------------------------------------------------- append_rope
CASES = [(None, [1, 16, 17, 40, 200]), ([1], [4]), ([5, 0, 17, 1, 64], [8, 20, 17, 16, 97]), ([700, 1, 300], [703, 21, 300])]


def positions_of(c):
    at = np.zeros(c["q"].shape[0], dtype=np.int64)
    starts = np.arange(len(c["lens"]) + 1) if c["starts"] is None else c["starts"]
    for b in range(len(c["lens"])):
        n = starts[b + 1] - starts[b]
        at[starts[b]:starts[b + 1]] = c["lens"][b] - n + np.arange(n)
    return at


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("q_heads,heads,dim,page,rot,interleaved", [
    (1, 1, 64, 16, 64, False), (6, 3, 96, 32, 24, False), (8, 8, 128, 64, 128, True), (32, 8, 128, 16, 128, False),
    (5, 1, 96, 16, 96, True), (4, 2, 256, 1024, 64, False), (0, 2, 128, 16, 40, True)])
@pytest.mark.parametrize("new,lens", CASES)
def test_append_rope_is_rope_and_append(env, dtype, q_heads, heads, dim, page, rot, interleaved, new, lens):
    torch, slim = env
    c = case(torch, 1, dtype, lens, heads, heads, dim, page, new=new)
    rope = slim.Rope(rot, interleaved=interleaved, scaling="yarn", factor=4.0, original_len=512)
    at = positions_of(c)
    k, v = c["q"], rows(torch, dtype, c["q"].shape[0], heads, dim, seed=3)
    q = rows(torch, dtype, k.shape[0], q_heads, dim, seed=4) if q_heads else None
    pools = [c["k"].clone(), c["v"].clone()]
    turned = slim.rope(k, ints(torch, at), rope)
    slim.kv_append(turned, v, *pools, c["d_table"], c["d_lens"], c["d_starts"])
    got = slim.kv_append_rope(k, v, c["k"], c["v"], c["d_table"], c["d_lens"], rope, starts=c["d_starts"], q=q)
    torch.cuda.synchronize()
    check(host(turned), host(k), at, rope, dtype, "keys")
    assert torch.equal(c["k"], pools[0]) and torch.equal(c["v"], pools[1])
    if q is None:
        assert got is None
    else:
        assert torch.equal(got, slim.rope(q, ints(torch, at), rope))
        check(host(got), host(q), at, rope, dtype, "queries")


def test_append_rope_strided_in_place_and_many_sequences(env):
    torch, slim = env
    rng = np.random.default_rng(2)
    new = [int(n) for n in rng.integers(0, 9, 3000)]
    c = case(torch, 2, "bf16", [n + int(p) for n, p in zip(new, rng.integers(0, 30, 3000))], 2, 2, 64, 16, new=new)
    rope = slim.Rope(32)
    joint = rows(torch, "bf16", c["q"].shape[0], 9, 64, seed=6)
    q, k, v = joint[:, :4], joint[:, 4:6], joint[:, 7:9]
    at = positions_of(c)
    want_q, turned = slim.rope(q, ints(torch, at), rope), slim.rope(k, ints(torch, at), rope)
    k0, v0 = host(c["k"]), host(c["v"])
    rest = joint[:, 4:].clone()
    slim.kv_append_rope(k, v, c["k"], c["v"], c["d_table"], c["d_lens"], rope, starts=c["d_starts"], q=q, q_out=q)
    torch.cuda.synchronize()
    rk, rv = attention_ref.append(host(turned), host(v), k0, v0, c["table"], c["lens"], c["starts"])
    assert np.array_equal(host(c["k"]), rk) and np.array_equal(host(c["v"]), rv)
    assert torch.equal(q, want_q) and torch.equal(joint[:, 4:], rest)


def test_append_rope_leaves_what_it_must_not_write(env):
    """Bad table entries, positions past the table, negative positions, rows before, between and past the batch."""
    torch, slim = env
    c = case(torch, 3, "fp16", [40, 64, 5, 30], 2, 2, 64, 16, new=[10, 4, 9, 3])
    c["table"][0, 2] = -1
    c["table"][3, 1] = c["k"].shape[0]
    c["lens"] = np.asarray([40, 66, 5, 30], dtype=np.int32)
    c["d_table"].copy_(torch.from_numpy(c["table"]))
    c["d_lens"].copy_(torch.from_numpy(c["lens"]))
    starts = c["starts"] + 7
    k, q = rows(torch, "fp16", 7 + 26 + 50, 2, 64), rows(torch, "fp16", 7 + 26 + 50, 4, 64, seed=2)
    rope = slim.Rope(64)
    k0, v0 = host(c["k"]), host(c["v"])
    out = torch.full_like(q, 77.0)
    slim.kv_append_rope(k, -k, c["k"], c["v"], c["d_table"], c["d_lens"], rope, starts=ints(torch, starts), q=q, q_out=out)
    torch.cuda.synchronize()
    at = np.concatenate([[0] * 7, positions_of(dict(c, starts=c["starts"])), [0] * 50])
    turned = slim.rope(k, ints(torch, at), rope)
    rk, rv = attention_ref.append(host(turned)[7:], host(-k)[7:], k0, v0, c["table"], c["lens"], c["starts"])
    assert np.array_equal(host(c["k"]), rk) and np.array_equal(host(c["v"]), rv)
    # Queries need no page: every row of a sequence is turned, also at positions without one.
    assert (out[:7] == 77).all() and (out[33:] == 77).all()
    assert torch.equal(out[7:33], slim.rope(q, ints(torch, at), rope)[7:33])


def test_append_rope_captured(env):
    torch, slim = env
    rope = slim.Rope(128)
    cs = [case(torch, 50 + i, "fp16", lens, 2, 2, 128, 16, new=[3, 20], width=80, pages=200)
          for i, lens in enumerate([[40, 700], [1000, 41], [20, 1280]])]
    st = {n: cs[0][n].clone() for n in ("q", "k", "v", "d_table", "d_lens")}
    queries = rows(torch, "fp16", 23, 8, 128)
    out = torch.empty_like(queries)

    def go(c, out):
        slim.kv_append_rope(c["q"], c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], rope, starts=cs[0]["d_starts"], q=queries,
                            q_out=out)

    go(st, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(st, out)
    for _ in range(2):
        for c in cs:
            for n in st:
                st[n].copy_(c[n])
            out.fill_(77.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            want, eager = torch.empty_like(out), {n: c[n].clone() for n in st}
            go(eager, want)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(st["k"], eager["k"]) and torch.equal(st["v"], eager["v"])


def test_append_rope_refusals_in_the_binding(env):
    torch, slim = env
    c = case(torch, 4, "fp16", [5, 9], 2, 2, 64, 16)
    rope, q = slim.Rope(64), rows(torch, "fp16", 2, 4, 64)
    good = dict(K=c["q"], V=c["q"], kpool=c["k"], vpool=c["v"], table=c["d_table"], lens=c["d_lens"], rope=rope)
    for bad in (dict(rope=None), dict(K=c["q"][:1]), dict(V=c["q"].bfloat16()), dict(q=q[:1]), dict(q=q, q_out=q[:, :2]),
                dict(q=q.float()), dict(kpool=c["k"].float()), dict(table=c["d_table"][:1]), dict(q_out=q),
                dict(q=rows(torch, "fp16", 2, 3, 64)), dict(kpool=c["k"].to(torch.uint8))):
        with pytest.raises((TypeError, ValueError, slim.SlimError)):
            slim.kv_append_rope(**{**good, **bad})

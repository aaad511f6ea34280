"""Rotations, appends and read-back of more rows than the processor holds waves
for at once (then a lane takes several vectors): against the oracle, and bit for
bit what the same rows give a few at a time."""
import numpy as np
import pytest

from oracle import q4_ref
from test_q4_gpu import env, turned  # noqa: F401
from test_rope_gpu import check, host, ints, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(2900, 33, 64, 64), (3001, 20, 80, 24), (8300, 5, 72, 72), (2050, 40, 128, 40),
                                                  (1100, 64, 256, 128), (4200, 31, 24, 8)])
def test_rope(env, dtype, interleaved, tokens, heads, dim, rot):
    torch, slim = env
    rope = slim.Rope(rot, interleaved=interleaved)
    x = rows(torch, dtype, tokens, heads, dim)
    at = np.random.default_rng(tokens).integers(0, 100000, tokens)
    y = slim.rope(x, ints(torch, at), rope)
    torch.cuda.synchronize()
    check(host(y), host(x), at, rope, dtype)
    for i in range(0, tokens, 97):
        assert torch.equal(slim.rope(x[i:i + 3], ints(torch, at[i:i + 3]), rope), y[i:i + 3])


# Tokens of three sequences (one of them has none) behind lengths that differ.
def layout(torch, tokens, heads, dim, page, pool):
    new = [tokens // 3, 0, tokens - tokens // 3]
    lens = [n + p for n, p in zip(new, (5, 33, 700))]
    width = max(-(-n // page) for n in lens)
    table = np.random.default_rng(tokens).permutation(3 * width + 2)[:3 * width].reshape(3, width)
    at = np.concatenate([np.arange(n - c, n) for n, c in zip(lens, new)])
    pools = [pool(3 * width + 2, heads, page, dim) for _ in range(2)]
    return pools, ints(torch, table), ints(torch, lens), ints(torch, np.cumsum([0, *new])), at


def few_at_a_time(torch, append, table, lens, starts, tokens):
    """append(first, last, table, lens, starts) on 50 tokens after the other."""
    starts, lens = starts.tolist(), lens.tolist()
    for i in range(0, tokens, 50):
        j = min(i + 50, tokens)
        part = [min(max(s, i), j) for s in starts]
        now = [n - max(0, s1 - max(j, s0)) for n, s0, s1 in zip(lens, starts, starts[1:])]
        append(i, j, table, ints(torch, now), ints(torch, [s - i for s in part]))


SHAPES = [(20, 20, 64, 16, 64, False), (9, 3, 96, 32, 24, True), (32, 8, 128, 64, 128, False), (0, 40, 96, 16, 96, False),
          (8, 4, 256, 128, 40, False), (0, 12, 128, 1024, 64, True)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("q_heads,heads,dim,page,rot,interleaved", SHAPES)
def test_append_rope(env, dtype, q_heads, heads, dim, page, rot, interleaved):
    torch, slim = env
    tokens = 4500
    rope = slim.Rope(rot, interleaved=interleaved)
    k, v = rows(torch, dtype, tokens, heads, dim), rows(torch, dtype, tokens, heads, dim, seed=2)
    q = rows(torch, dtype, tokens, q_heads, dim, seed=3) if q_heads else None
    pools, table, lens, starts, at = layout(torch, tokens, heads, dim, page,
                                            lambda *s: torch.full(s, 77.0, device="cuda", dtype=k.dtype))
    parts = [p.clone() for p in pools]
    got = slim.kv_append_rope(k, v, *pools, table, lens, rope, starts=starts, q=q)
    few_at_a_time(torch, lambda i, j, t, n, s: slim.kv_append_rope(k[i:j], v[i:j], *parts, t, n, rope, starts=s),
                  table, lens, starts, tokens)
    plain = [torch.full_like(p, 77.0) for p in pools]
    slim.kv_append(slim.rope(k, ints(torch, at), rope), v, *plain, table, lens, starts)
    torch.cuda.synchronize()
    for a, b, c in zip(pools, parts, plain):
        assert torch.equal(a, b) and torch.equal(a, c)
    if q_heads:
        check(host(got), host(q), at, rope, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("q_heads,heads,dim,page,rot,interleaved", [*SHAPES, (0, 33, 64, 16, 0, False)])
def test_append_and_read_q4(env, dtype, q_heads, heads, dim, page, rot, interleaved):
    torch, slim = env
    tokens = 4500
    rope = slim.Rope(rot, interleaved=interleaved) if rot else None
    k, v = rows(torch, dtype, tokens, heads, dim), rows(torch, dtype, tokens, heads, dim, seed=2)
    q = rows(torch, dtype, tokens, q_heads, dim, seed=3) if q_heads else None
    pools, table, lens, starts, at = layout(torch, tokens, heads, dim, page, lambda p, h, s, d: torch.full(
        (p, h, s, d * 17 // 32), 0x5A, device="cuda", dtype=torch.uint8))
    parts = [p.clone() for p in pools]
    got = slim.kv_append_q4(k, v, *pools, table, lens, starts=starts, rope=rope, q=q)
    few_at_a_time(torch, lambda i, j, t, n, s: slim.kv_append_q4(k[i:j], v[i:j], *parts, t, n, starts=s, rope=rope),
                  table, lens, starts, tokens)
    out = [torch.full((tokens + 9, heads, dim), 77.0, device="cuda", dtype=k.dtype) for _ in range(2)]
    slim.kv_read_q4(*pools, table, lens, starts=starts + 4, out=tuple(out))
    torch.cuda.synchronize()
    assert torch.equal(pools[0], parts[0]) and torch.equal(pools[1], parts[1])
    for o, x in zip(out, (turned(host(k), at, rope) if rope else host(k), host(v))):
        assert np.array_equal(host(o[4:-5]), q4_ref.decode(*q4_ref.encode(x, dtype)))
        assert (o[:4] == 77).all() and (o[-5:] == 77).all()
    if q_heads:
        check(host(got), host(q), at, rope, dtype)

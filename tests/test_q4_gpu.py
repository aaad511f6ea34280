"""slim_kv_append_q4 and slim_kv_read_q4 against the oracle, byte for byte:
types, layouts, turned and plain keys, borders between codes, values at the ends
of the types, infinities, and bytes that must stay; pages copied, forked and compacted."""
import numpy as np
import pytest

from attention_helpers import case, host
from oracle import q4_ref, rope_ref
from q4_helpers import q4_case
from test_rope_gpu import CASES, ints, positions_of, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


def turned(k, at, rope):
    """Turned keys as they are coded: held in fp32."""
    return rope_ref.turn(k, at, rope.freqs.cpu().numpy(), rope.interleaved, rope.magnitude).astype(np.float32)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("q_heads,heads,dim,page,rot,interleaved", [
    (0, 1, 64, 16, 0, False), (6, 3, 96, 32, 24, False), (8, 8, 128, 64, 128, True), (32, 8, 128, 16, 128, False),
    (5, 1, 96, 16, 96, True), (4, 2, 256, 1024, 64, False), (0, 2, 128, 16, 40, True), (0, 20, 96, 16, 0, False)])
@pytest.mark.parametrize("new,lens", CASES)
def test_append_and_read(env, dtype, q_heads, heads, dim, page, rot, interleaved, new, lens):
    """Every byte of both pools as the oracle has it, the others as they were.  (Codes are chosen by keys turned in
    fp64 here and there, which differ by some 2^-50; of a million random ones none lies so near a border.)"""
    torch, slim = env
    c = q4_case(torch, 1, dtype, lens, heads, heads, dim, page, new=new)
    rope = slim.Rope(rot, interleaved=interleaved, scaling="linear", factor=2.0) if rot else None
    at = positions_of(c)
    k = c["q"]
    v = rows(torch, dtype, k.shape[0], heads, dim, seed=3) * torch.exp2(torch.arange(dim, device="cuda") % 7 - 3).to(k.dtype)
    q = rows(torch, dtype, k.shape[0], q_heads, dim, seed=4) if q_heads else None
    k4, v4 = c["k4"].cpu().numpy(), c["v4"].cpu().numpy()
    got = slim.kv_append_q4(k, v, c["k4"], c["v4"], c["d_table"], c["d_lens"], starts=c["d_starts"], rope=rope, q=q)
    torch.cuda.synchronize()
    as_coded = turned(host(k), at, rope) if rope else host(k)
    rk, rv = q4_ref.append(as_coded, host(v), k4, v4, c["table"], c["lens"], c["starts"], dtype)
    assert np.array_equal(c["k4"].cpu().numpy(), rk) and np.array_equal(c["v4"].cpu().numpy(), rv)
    assert got is None if q is None else torch.equal(got, slim.rope(q, ints(torch, at), rope))
    # Read back: exactly what the codes stand for.
    kr, vr = slim.kv_read_q4(c["k4"], c["v4"], c["d_table"], c["d_lens"], starts=c["d_starts"], tokens=k.shape[0], dtype=k.dtype)
    torch.cuda.synchronize()
    assert np.array_equal(host(kr), q4_ref.decode(*q4_ref.encode(as_coded, dtype)))
    assert np.array_equal(host(vr), q4_ref.decode(*q4_ref.encode(host(v), dtype)))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_every_half_value(env, dtype):
    """Every finite value of the type, as its group's largest and beside larger ones: scales and codes at all borders, ties
    among them, at both ends of the range and at zeros."""
    torch, slim = env
    every = torch.arange(-2 ** 15, 2 ** 15, device="cuda", dtype=torch.int32).to(torch.int16).view(
        torch.float16 if dtype == "fp16" else torch.bfloat16)
    every = every[every.isfinite()]
    n = every.numel()
    k = torch.zeros((n // 8 + 1, 8, 128), dtype=every.dtype, device="cuda").view(-1, 128)[:n].contiguous()
    k[:, 5] = every                                       # alone
    k[:, 32:64] = every[:, None] * torch.linspace(0, 1, 32, device="cuda").to(every.dtype)
    k[:, 64:96] = every[:, None]
    k[:, 96:] = every[torch.randperm(n, device="cuda", generator=torch.Generator("cuda").manual_seed(1))][:, None]
    k[:, 100] = every                                     # beside others of any size
    k = k.view(n, 1, 128)
    table = torch.arange(-(-n // 1024), device="cuda", dtype=torch.int32)[None]
    pool = [torch.full((table.shape[1], 1, 1024, 68), 0xAA, dtype=torch.uint8, device="cuda") for _ in range(2)]
    at, starts = ints(torch, [n]), ints(torch, [0, n])
    slim.kv_append_q4(k, k.flip(0), *pool, table, at, starts=starts)
    kr, vr = slim.kv_read_q4(*pool, table, at, starts=starts, tokens=n, dtype=k.dtype)
    torch.cuda.synchronize()
    code, scale = q4_ref.encode(host(k), dtype)
    got_code, got_scale = q4_ref.unpack(pool[0].cpu().numpy())
    assert np.array_equal(got_code.reshape(-1, 128)[:n], code[:, 0]) and np.array_equal(got_scale.reshape(-1, 4)[:n], scale[:, 0])
    want = q4_ref.decode(code, scale)
    assert np.isfinite(host(kr)).all() and np.array_equal(host(kr), want) and np.array_equal(host(vr), want[::-1])


def test_turned_keys_next_to_borders(env):
    """Rows scaled so that one turned element of a group lies as near 2.5 as fp16 inputs allow, the group's scale being 1."""
    torch, slim = env
    rope = slim.Rope(128)
    n = 4000
    at = np.random.default_rng(9).integers(0, 16, n)          # each token in a page of its own sequence
    k = rows(torch, "fp16", n, 2, 128, seed=9)
    t = rope_ref.turn(host(k), at, rope.freqs.cpu().numpy())
    j = np.arange(n) % 32
    by = 2.5 / np.maximum(np.abs(t[np.arange(n), 0, j]), 0.4)
    k[:, 0] = k[:, 0] * torch.from_numpy(by).cuda().half()[:, None]
    pool = [torch.zeros((n, 2, 16, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.arange(n, device="cuda", dtype=torch.int32)[:, None].contiguous()
    slim.kv_append_q4(k, k, *pool, table, ints(torch, at + 1), rope=rope)
    torch.cuda.synchronize()
    code, scale = q4_ref.encode(turned(host(k), at, rope), "fp16")
    got_code, got_scale = q4_ref.unpack(pool[0].cpu().numpy())
    i = np.arange(n)
    assert np.array_equal(got_code[i, :, at], code) and np.array_equal(got_scale[i, :, at], scale)


def test_infinities_and_nan_make_their_group_nan(env):
    torch, slim = env
    k = rows(torch, "bf16", 4, 2, 96, seed=2)
    k[0, 0, 3], k[1, 1, 95], k[2, 0, 40] = float("nan"), float("inf"), -float("inf")
    pool = [torch.zeros((4, 2, 16, 51), dtype=torch.uint8, device="cuda") for _ in range(2)]
    table, lens = ints(torch, [[0], [1], [2], [3]]), ints(torch, [1, 5, 16, 7])
    for rope in (None, slim.Rope(32)):
        slim.kv_append_q4(k, k, *pool, table, lens, rope=rope)
        kr, vr = slim.kv_read_q4(*pool, table, lens, dtype=k.dtype)
        torch.cuda.synchronize()
        bad = np.zeros((4, 2, 96), dtype=bool)
        bad[0, 0, :32] = bad[1, 1, 64:] = bad[2, 0, 32:64] = True
        assert np.array_equal(np.isnan(host(vr)), bad) and np.array_equal(np.isnan(host(kr)), bad)
    code, scale = q4_ref.unpack(pool[1].cpu().numpy())
    assert scale[0, 0, 0, 0] == 255 and not code[0, 0, 0, :32].any() and (scale[0, 1] != 255).all()


def test_what_is_not_written_and_not_read(env):
    """Bad table entries, positions past the table, negative ones, rows before and past the batch: no byte of a pool but the
    new rows' changes; rows without a page read as zeros, rows of no sequence stay."""
    torch, slim = env
    c = q4_case(torch, 3, "fp16", [40, 64, 5, 30], 2, 2, 64, 16, new=[10, 4, 9, 3])
    c["table"][0, 2] = -1
    c["table"][3, 1] = c["k"].shape[0]
    c["lens"] = np.asarray([40, 66, 5, 30], dtype=np.int32)
    c["d_table"].copy_(torch.from_numpy(c["table"]))
    c["d_lens"].copy_(torch.from_numpy(c["lens"]))
    k = rows(torch, "fp16", 7 + 26 + 50, 2, 64)
    k4, v4 = c["k4"].cpu().numpy(), c["v4"].cpu().numpy()
    starts = ints(torch, c["starts"] + 7)
    slim.kv_append_q4(k, -k, c["k4"], c["v4"], c["d_table"], c["d_lens"], starts=starts)
    out = [torch.full_like(k, 77.0) for _ in range(2)]
    slim.kv_read_q4(c["k4"], c["v4"], c["d_table"], c["d_lens"], starts=starts, out=tuple(out))
    torch.cuda.synchronize()
    rk, rv = q4_ref.append(host(k)[7:], host(-k)[7:], k4, v4, c["table"], c["lens"], c["starts"], "fp16")
    assert np.array_equal(c["k4"].cpu().numpy(), rk) and np.array_equal(c["v4"].cpu().numpy(), rv)
    want = q4_ref.decode(*q4_ref.encode(host(k), "fp16"))
    at, page = positions_of(c), np.repeat(np.arange(4), np.diff(c["starts"]))
    for t in range(26):
        b, p = page[t], at[t]
        there = 0 <= p < 64 and 0 <= c["table"][b, p // 16] < c["k"].shape[0]
        assert np.array_equal(host(out[0])[7 + t], want[7 + t] if there else np.zeros((2, 64)))
        assert np.array_equal(host(out[1])[7 + t], -want[7 + t] if there else np.zeros((2, 64)))
    for o in out:
        assert (o[:7] == 77).all() and (o[33:] == 77).all()


def test_strided_rows_streams_and_graph(env):
    torch, slim = env
    c = q4_case(torch, 5, "bf16", [33, 100, 64], 2, 2, 96, 16, new=[33, 5, 64])
    rope = slim.Rope(96, interleaved=True)
    joint = rows(torch, "bf16", 102, 9, 96, seed=6)
    q, k, v = joint[:, :4], joint[:, 4:6], joint[:, 7:9]
    want = [c["k4"].clone(), c["v4"].clone()]
    want_q = slim.kv_append_q4(k.contiguous(), v.contiguous(), *want, c["d_table"], c["d_lens"], starts=c["d_starts"], rope=rope,
                               q=q.contiguous())
    pool = [c["k4"].clone(), c["v4"].clone()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = slim.kv_append_q4(k, v, *pool, c["d_table"], c["d_lens"], starts=c["d_starts"], rope=rope, q=q, stream=side)
    wide = torch.full((102, 5, 96), 77.0, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    slim.kv_read_q4(*pool, c["d_table"], c["d_lens"], starts=c["d_starts"], out=(wide[:, :2], wide[:, 3:]))
    kr, vr = slim.kv_read_q4(*want, c["d_table"], c["d_lens"], starts=c["d_starts"], tokens=102, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pool, want)) and torch.equal(got, want_q)
    assert torch.equal(wide[:, :2], kr) and torch.equal(wide[:, 3:], vr) and (wide[:, 2] == 77).all()
    pool = [c["k4"].clone(), c["v4"].clone()]
    out = torch.empty_like(want_q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slim.kv_append_q4(k, v, *pool, c["d_table"], c["d_lens"], starts=c["d_starts"], rope=rope, q=q, q_out=out)
    for turn in range(3):
        joint.copy_(rows(torch, "bf16", 102, 9, 96, seed=60 + turn))
        eager = [p.clone() for p in pool]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager_q = slim.kv_append_q4(k, v, *eager, c["d_table"], c["d_lens"], starts=c["d_starts"], rope=rope, q=q)
        assert all(torch.equal(a, b) for a, b in zip(pool, eager)) and torch.equal(out, eager_q)


def test_cache_of_four_bits_forks_copies_and_compacts(env):
    """Appends, a fork, a free and a compaction: every sequence reads back its own history."""
    torch, slim = env
    cache = slim.KVCache(2, 40, 2, 64, page_size=16, dtype=torch.bfloat16, bits=4)
    cache.k.fill_(0xFF)
    cache.v.fill_(0xFF)
    rng = np.random.default_rng(8)
    history: dict[int, list] = {}

    def step(seqs, counts):
        batch = cache.extend(seqs, counts)
        new = rows(torch, "bf16", sum(counts), 2, 64, seed=int(rng.integers(1 << 30)))
        for layer in range(2):
            slim.kv_append_q4(new * (layer + 1), new - 1, cache.k[layer], cache.v[layer], batch.table, batch.lens,
                              starts=batch.starts)
        at = 0
        for s, n in zip(seqs, counts):
            history[s] += list(new[at:at + n])
            at += n

    def check():
        for s, h in history.items():
            if not h:
                continue
            n = len(h)
            batch, x = cache.batch([s], [n]), torch.stack(h)
            for layer in range(2):
                k, v = slim.kv_read_q4(cache.k[layer], cache.v[layer], batch.table, batch.lens, starts=batch.starts, tokens=n,
                                       dtype=torch.bfloat16)
                torch.cuda.synchronize()
                assert np.array_equal(host(k), q4_ref.decode(*q4_ref.encode(host(x * (layer + 1)), "bf16")))
                assert np.array_equal(host(v), q4_ref.decode(*q4_ref.encode(host(x - 1), "bf16")))

    a, b = cache.add(), cache.add()
    history.update({a: [], b: []})
    step([a, b], [37, 20])
    f = cache.fork(a)
    history[f] = list(history[a])
    step([a, f, b], [3, 1, 30])
    check()
    cache.free(a)
    del history[a]
    assert cache.compact() > 0
    step([f, b], [18, 1])
    check()


def test_a_long_cache_passes_32_bits(env):
    """Pages whose byte offsets pass 2^31 and 2^32."""
    torch, slim = env
    heads, page, dim = 8, 64, 128
    pages = (5 << 30) // slim.slim_q4_page_bytes(heads, page, dim)
    pools = [torch.empty((pages, heads, page, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    far = [0, pages // 2, pages - 3, pages - 1]
    k = rows(torch, "fp16", 4 * 64, heads, dim)
    table, lens, starts = ints(torch, [[p] for p in far]), ints(torch, [64] * 4), ints(torch, [0, 64, 128, 192, 256])
    slim.kv_append_q4(k, -k, *pools, table, lens, starts=starts)
    kr, vr = slim.kv_read_q4(*pools, table, lens, starts=starts, tokens=256)
    near = [torch.zeros((4, heads, page, 68), dtype=torch.uint8, device="cuda") for _ in range(2)]
    slim.kv_append_q4(k, -k, *near, ints(torch, [[0], [1], [2], [3]]), lens, starts=starts)
    torch.cuda.synchronize()
    for i, p in enumerate(far):
        assert torch.equal(pools[0][p], near[0][i]) and torch.equal(pools[1][p], near[1][i])
    want = q4_ref.decode(*q4_ref.encode(host(k), "fp16"))
    assert np.array_equal(host(kr), want) and np.array_equal(host(vr), -want)
    # And the attention over them.
    q = rows(torch, "fp16", 40, 16, dim, seed=3)
    near_table, qs = ints(torch, [[0], [1], [2], [3]]), ints(torch, [0, 33, 34, 40, 40])
    assert torch.equal(slim.attention_decode_q4(q[:4], *pools, table, lens), slim.attention_decode_q4(q[:4], *near, near_table, lens))
    assert torch.equal(slim.attention_prefill_q4(q, *pools, table, lens, qs), slim.attention_prefill_q4(q, *near, near_table, lens, qs))


def test_refusals_in_the_binding(env):
    torch, slim = env
    c = q4_case(torch, 4, "fp16", [5, 9], 2, 2, 64, 16)
    rope, q = slim.Rope(64), rows(torch, "fp16", 2, 4, 64)
    good = dict(K=c["q"], V=c["q"], kpool=c["k4"], vpool=c["v4"], table=c["d_table"], lens=c["d_lens"])
    for bad in (dict(K=c["q"][:1]), dict(V=c["q"].bfloat16()), dict(K=c["q"].float()), dict(q=q), dict(q=q[:1], rope=rope),
                dict(kpool=c["k"]), dict(kpool=c["k4"][..., :33]), dict(vpool=c["v4"][:1]), dict(kpool=c["k4"].cpu()),
                dict(table=c["d_table"].long()), dict(rope=slim.Rope(96)), dict(starts=ints(torch, [0, 2]))):
        with pytest.raises((TypeError, ValueError, slim.SlimError)):
            slim.kv_append_q4(**{**good, **bad})
    pools = dict(kpool=c["k4"], vpool=c["v4"], table=c["d_table"], lens=c["d_lens"])
    for bad in (dict(starts=ints(torch, [0, 1, 2])), dict(dtype=torch.float32), dict(tokens=3), dict(out=(c["q"], c["q"][:1])),
                dict(kpool=c["k"])):
        with pytest.raises((TypeError, ValueError, slim.SlimError)):
            slim.kv_read_q4(**{**pools, **bad})

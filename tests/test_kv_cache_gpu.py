"""slim_kv_append and slim_kv_copy_pages against the oracle (exact), and the
paged cache end to end: appends, forks, frees, drops and compaction leave every
sequence's attention as the oracle has it on the sequence's own history."""
import numpy as np
import pytest

from attention_helpers import bound, case, host
from oracle import attention_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (3, 96, 32), (8, 128, 64), (32, 128, 16), (2, 256, 1024)])
@pytest.mark.parametrize("new", [None, [1], [5, 0, 17, 1, 64], [700, 1, 300]])
def test_append(env, dtype, heads, dim, page, new):
    torch, slim = env
    lens = [1, 16, 17, 40, 200] if new is None else [n + p for n, p in zip(new, [3, 20, 0, 15, 33])]
    c = case(torch, 1, dtype, lens, heads, heads, dim, page, new=new)
    k_new = c["q"]
    v_new = (c["q"] * 0.5 + 1).contiguous()
    k0, v0 = host(c["k"]), host(c["v"])
    slim.kv_append(k_new, v_new, c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"])
    torch.cuda.synchronize()
    rk, rv = ref.append(host(k_new), host(v_new), k0, v0, c["table"], c["lens"], c["starts"])
    assert np.array_equal(host(c["k"]), rk) and np.array_equal(host(c["v"]), rv)


def test_append_many_sequences_and_strided_rows(env):
    torch, slim = env
    rng = np.random.default_rng(2)
    new = [int(n) for n in rng.integers(0, 9, 5000)]
    c = case(torch, 2, "bf16", [n + int(p) for n, p in zip(new, rng.integers(0, 30, 5000))], 2, 2, 64, 16, new=new)
    joint = torch.randn(c["q"].shape[0], 9, 64, device="cuda").bfloat16()
    k0, v0 = host(c["k"]), host(c["v"])
    slim.kv_append(joint[:, 4:6], joint[:, 7:9], c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"])
    torch.cuda.synchronize()
    rk, rv = ref.append(host(joint[:, 4:6]), host(joint[:, 7:9]), k0, v0, c["table"], c["lens"], c["starts"])
    assert np.array_equal(host(c["k"]), rk) and np.array_equal(host(c["v"]), rv)


def test_append_leaves_what_it_must_not_write(env):
    """Bad table entries, positions past the table, negative positions, rows past the batch."""
    torch, slim = env
    c = case(torch, 3, "fp16", [40, 64, 5, 30], 2, 2, 64, 16, new=[10, 4, 9, 3])
    c["table"][0, 2] = -1
    c["table"][3, 1] = c["k"].shape[0]
    c["lens"] = np.asarray([40, 66, 5, 30], dtype=np.int32)
    c["d_table"].copy_(torch.from_numpy(c["table"]))
    c["d_lens"].copy_(torch.from_numpy(c["lens"]))
    rows = torch.randn(26 + 50, 2, 64, device="cuda").half()
    k0, v0 = host(c["k"]), host(c["v"])
    slim.kv_append(rows, rows, c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"])
    torch.cuda.synchronize()
    rk, rv = ref.append(host(rows), host(rows), k0, v0, c["table"], c["lens"], c["starts"])
    assert np.array_equal(host(c["k"]), rk) and np.array_equal(host(c["v"]), rv)
    for s in ([-5, 40, 10 ** 6, 3, 2], [30, 20, 10, 0, -1], [10 ** 6] * 5, [-2 ** 31, 0, 0, 0, 2 ** 31 - 1]):
        slim.kv_append(rows, rows, c["k"], c["v"], c["d_table"], c["d_lens"],
                       torch.tensor(s, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()


@pytest.mark.parametrize("layers,heads,page,dim", [(1, 1, 16, 64), (3, 2, 16, 96), (2, 8, 64, 128), (2, 5, 1024, 64)])
def test_copy_pages(env, layers, heads, page, dim):
    torch, slim = env
    k = torch.randn(layers, 12, heads, page, dim, device="cuda").half()
    v = torch.randn(layers, 12, heads, page, dim, device="cuda").half()
    src, dst = [3, 0, 3, -1, 5, 12, 2 ** 31 - 1], [7, 1, 11, 4, 12, 6, 8]
    k0, v0 = host(k), host(v)
    slim.kv_copy_pages(k, v, torch.tensor(src, dtype=torch.int32, device="cuda"),
                       torch.tensor(dst, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(host(k), ref.copy_pages(k0, src, dst)) and np.array_equal(host(v), ref.copy_pages(v0, src, dst))
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    slim.kv_copy_pages(k, v, empty, empty)


def test_cache_serves_forks_frees_and_compaction(env):
    """A serving run on two layers; the host keeps each sequence's own keys and values."""
    torch, slim = env
    layers, kv_heads, q_heads, dim, page = 2, 2, 4, 64, 16
    cache = slim.KVCache(layers, 40, kv_heads, dim, page_size=page, dtype=torch.float16)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    past: dict[int, list] = {}

    def step(ids, counts):
        batch = cache.extend(ids, counts)
        rows = [torch.randn(batch.tokens, h, dim, generator=gen, device="cuda").half() for h in (q_heads, kv_heads, kv_heads)]
        for layer in range(layers):
            k, v = rows[1] * (layer + 1), rows[2] + layer
            slim.kv_append(k, v, cache.k[layer], cache.v[layer], batch.table, batch.lens, batch.starts)
            out = slim.attention_prefill(rows[0], cache.k[layer], cache.v[layer], batch.table, batch.lens, batch.starts,
                                         max_len=batch.max_len)
            if all(c == 1 for c in counts):
                one = slim.attention_decode(rows[0], cache.k[layer], cache.v[layer], batch.table, batch.lens)
            at = 0
            for q, c in zip(ids, counts):
                hist = past[q][layer]
                hist[0] = np.concatenate([hist[0], host(k[at:at + c])])
                hist[1] = np.concatenate([hist[1], host(v[at:at + c])])
                n = hist[0].shape[0]
                args = (host(rows[0][at:at + c]), hist[0].transpose(1, 0, 2)[None], hist[1].transpose(1, 0, 2)[None],
                        np.zeros((1, 1), dtype=np.int32), [n], [0, c], dim ** -0.5)
                want, _, mass = ref.attention(*args)
                for y in (out,) + ((one,) if all(c == 1 for c in counts) else ()):
                    over = np.abs(host(y[at:at + c]) - want) - bound(dict(dtype="fp16"), want, mass)
                    assert over.max(initial=-1) <= 0, (q, layer, over.max())
                at += c

    def new():
        q = cache.add()
        past[q] = [[np.zeros((0, kv_heads, dim)), np.zeros((0, kv_heads, dim))] for _ in range(layers)]
        return q

    def fork(q):
        f = cache.fork(q)
        past[f] = [[a.copy(), b.copy()] for a, b in past[q]]
        return f

    a, b = new(), new()
    step([a, b], [37, 16])
    step([a, b], [1, 1])
    c = fork(a)                              # shares a part-filled page
    d = fork(b)
    step([a, c, d], [1, 1, 1])               # a and d take copies
    step([b, c], [20, 3])
    cache.free(a)
    e = fork(c)
    step([e, c, d, b], [1, 1, 1, 1])
    cache.free(b)
    moved = cache.compact()
    assert moved > 0
    used = {p for q in (c, d, e) for p in cache.pages(q)}
    assert used == set(range(len(used))) and cache.free_pages == 40 - len(used)
    step([c, e, d], [2, 1, 30])
    step([c, e, d], [1, 1, 1])
    before = (cache.free_pages, [cache.pages(q) for q in (c, d, e)])
    with pytest.raises(slim.CacheFull):
        cache.extend([c, d], [1, 100000])
    assert before == (cache.free_pages, [cache.pages(q) for q in (c, d, e)])
    for q in (c, d, e):
        cache.free(q)
    assert cache.free_pages == 40


def test_dropped_pages_of_a_windowed_sequence(env):
    torch, slim = env
    cache = slim.KVCache(1, 30, 1, 64, page_size=16)
    q = cache.add()
    window, sinks = 50, 4
    batch = cache.extend([q], [300])
    rows = torch.randn(300, 1, 64, device="cuda").half()
    slim.kv_append(rows, rows, cache.k[0], cache.v[0], batch.table, batch.lens, batch.starts)
    x = torch.randn(1, 2, 64, device="cuda").half()
    kept = [cache.extend([q]) for _ in range(1)][0]
    slim.kv_append(rows[:1], rows[:1], cache.k[0], cache.v[0], kept.table, kept.lens)
    want = slim.attention_decode(x, cache.k[0], cache.v[0], kept.table, kept.lens, window=window, sinks=sinks)
    cache.k[0, cache.pages(q)[5]].fill_(float("nan"))       # not seen any more
    assert cache.drop(q, window, sinks) == (301 - window + 1) // 16 - 1
    assert cache.pages(q)[0] >= 0 and cache.pages(q)[1] == -1
    batch = cache.batch([q])
    got = slim.attention_decode(x, cache.k[0], cache.v[0], batch.table, batch.lens, window=window, sinks=sinks)
    assert torch.equal(got, want)

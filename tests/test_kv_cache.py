"""The paged cache's bookkeeping, on the host: pages are owned by exactly the
sequences that list them, forks copy on their first write, nothing leaks."""
import random

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def slim(monkeypatch):
    import sparse_int4_gemm_amd as slim
    from sparse_int4_gemm_amd import _lib

    def copy(k, v, src, dst, stream=None):
        assert not set(src.tolist()) & set(dst.tolist()) and len(set(dst.tolist())) == dst.numel()
        for pool in (k, v):
            pool[:, dst.long()] = pool[:, src.long()]

    monkeypatch.setattr(_lib, "slim_kv_copy_pages", copy)
    return slim


def check(cache, ids):
    owners = [0] * cache.k.shape[1]
    for q in ids:
        pages = cache.pages(q)
        assert len(pages) == -(-cache.length(q) // cache.page_size)
        for p in pages:
            if p >= 0:
                owners[p] += 1
    assert owners == cache._owners
    assert sorted(cache._free) == [p for p, n in enumerate(owners) if n == 0]


def write(cache, batch, ids, counts, stamp, history):
    for b, (q, c) in enumerate(zip(ids, counts)):
        n = int(batch.lens[b])
        assert n == cache.length(q)
        for i in range(n - c, n):
            page = int(batch.table[b, i // cache.page_size])
            cache.k[:, page, :, i % cache.page_size] = stamp
            history[q].append(stamp)
            stamp += 1
    return stamp


def test_random_use_keeps_every_history(slim):
    rng = random.Random(5)
    cache = slim.KVCache(1, 24, 1, 1, page_size=4, dtype=torch.float32, device="cpu")
    history, stamp, full = {}, 1, 0
    for _ in range(600):
        ids = list(history)
        act = rng.choice(("add", "fork", "free", "extend", "extend", "extend", "compact"))
        if act == "add" and len(ids) < 6:
            history[cache.add()] = []
        elif act == "fork" and ids and len(ids) < 8:
            q = rng.choice(ids)
            history[cache.fork(q)] = list(history[q])
        elif act == "free" and len(ids) > 2:
            q = rng.choice(ids)
            cache.free(q)
            del history[q]
        elif act == "compact":
            cache.compact()
            live = 24 - cache.free_pages
            assert all(p < live for q in ids for p in cache.pages(q))
        elif act == "extend" and ids:
            some = rng.sample(ids, rng.randint(1, len(ids)))
            counts = [rng.randint(0, 5) for _ in some]
            try:
                batch = cache.extend(some, counts)
            except slim.CacheFull:
                full += 1
            else:
                assert batch.tokens == sum(counts) and batch.starts.tolist()[-1] == sum(counts)
                stamp = write(cache, batch, some, counts, stamp, history)
        check(cache, list(history))
        for q, h in history.items():
            pages = cache.pages(q)
            got = [float(cache.k[0, pages[i // 4], 0, i % 4, 0]) for i in range(len(h))]
            assert got == h
    assert full > 0


def test_refusals(slim):
    cache = slim.KVCache(1, 4, 1, 1, page_size=4, dtype=torch.float32, device="cpu")
    q = cache.add()
    with pytest.raises(ValueError):
        cache.extend([q, q])
    with pytest.raises(ValueError):
        cache.extend([q], [-1])
    with pytest.raises(ValueError):
        cache.extend([q], [1, 2])
    with pytest.raises(KeyError):
        cache.extend([99])
    with pytest.raises(slim.CacheFull):
        cache.extend([q], [17])
    assert cache.length(q) == 0 and cache.free_pages == 4
    with pytest.raises(ValueError):
        cache.drop(q, 0)
    with pytest.raises(ValueError):
        slim.KVCache(0, 4, 1, 1, device="cpu")
    cache.free(q)
    with pytest.raises(KeyError):
        cache.free(q)


def test_drop_keeps_what_a_window_sees(slim):
    cache = slim.KVCache(1, 16, 1, 1, page_size=4, dtype=torch.float32, device="cpu")
    q = cache.add()
    cache.extend([q], [30])
    f = cache.fork(q)
    # The next token, 30, sees 21 .. 30 and 0 .. 4: pages 0, 1 and from 5 (20 .. 23) on stay.
    assert cache.drop(q, 10, 5) == 3
    assert [p >= 0 for p in cache.pages(q)] == [True, True, False, False, False, True, True, True]
    assert cache.free_pages == 8                # the fork owns them still
    assert cache.drop(q, 10, 5) == 0
    cache.free(f)
    assert cache.free_pages == 11
    check(cache, [q])
    cache.compact()
    check(cache, [q])
    cache.extend([q], [3])
    assert cache.drop(q, 1) == 5 and cache.length(q) == 33        # 33 sees itself only: 0, 1, 5, 6, 7 go
    check(cache, [q])

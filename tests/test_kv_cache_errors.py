"""An error while pages are copied or the batch is made leaves the cache as it
was: no page lost, shared pages still shared, the same tokens in every sequence."""
import random

import pytest

torch = pytest.importorskip("torch")


class Broken(RuntimeError):
    pass


@pytest.fixture
def cache(monkeypatch):
    import sparse_int4_gemm_amd as slim
    from sparse_int4_gemm_amd import _lib
    cache = slim.KVCache(1, 24, 1, 1, page_size=4, dtype=torch.float32, device="cpu")
    cache.fails = None

    def copy(k, v, src, dst, stream=None):
        if cache.fails == "copy":
            raise Broken
        for pool in (k, v):
            pool[:, dst.long()] = pool[:, src.long()]

    batch = cache.batch

    def make(*args):
        if cache.fails == "batch":
            raise Broken
        return batch(*args)

    monkeypatch.setattr(_lib, "slim_kv_copy_pages", copy)
    monkeypatch.setattr(cache, "batch", make)
    return cache


def state(cache):
    return {q: (cache.pages(q), cache.length(q)) for q in cache._seqs}, list(cache._owners), sorted(cache._free)


@pytest.mark.parametrize("where", ["copy", "batch"])
def test_extend(cache, where):
    a = cache.add()
    cache.extend([a], [6])
    b, c = cache.fork(a), cache.fork(a)
    d = cache.add()
    before = state(cache)
    cache.fails = where
    for _ in range(3):
        with pytest.raises(Broken):
            cache.extend([a, b, d, c], [5, 1, 9, 2])
        assert state(cache) == before
    cache.fails = None
    batch = cache.extend([a, b, d, c], [5, 1, 9, 2])
    assert batch.lens.tolist() == [11, 7, 9, 8]
    last = [cache.pages(q)[1] for q in (a, b, c)]
    assert len(set(last)) == 3 and len({cache.pages(q)[0] for q in (a, b, c)}) == 1


def test_compact(cache):
    ids = [cache.add() for _ in range(4)]
    for q in ids:
        cache.extend([q], [9])
    cache.free(ids[0])
    cache.free(ids[2])
    before = state(cache)
    cache.fails = "copy"
    with pytest.raises(Broken):
        cache.compact()
    assert state(cache) == before
    cache.fails = None
    assert cache.compact() == 3
    assert sorted(p for q in (ids[1], ids[3]) for p in cache.pages(q)) == list(range(6))


def test_random_errors_between_random_use(cache):
    rng = random.Random(7)
    history, stamp = {}, 1
    for _ in range(500):
        ids = list(history)
        act = rng.choice(("add", "fork", "free", "extend", "extend", "extend", "compact"))
        cache.fails = rng.choice((None, None, "copy", "batch"))
        before = state(cache)
        try:
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
            elif act == "extend" and ids:
                some = rng.sample(ids, rng.randint(1, len(ids)))
                counts = [rng.randint(0, 5) for _ in some]
                batch = cache.extend(some, counts)
                for b, (q, c) in enumerate(zip(some, counts)):
                    for i in range(cache.length(q) - c, cache.length(q)):
                        cache.k[:, int(batch.table[b, i // 4]), :, i % 4] = stamp
                        history[q].append(stamp)
                        stamp += 1
        except RuntimeError:                     # Broken or CacheFull
            assert state(cache) == before
        for q, h in history.items():
            pages = cache.pages(q)
            assert [float(cache.k[0, pages[i // 4], 0, i % 4, 0]) for i in range(len(h))] == h

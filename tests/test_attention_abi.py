"""The attention and cache entry points refuse what they cannot do before they
touch a device, at the C boundary and in the binding."""
import pytest

P = 0x10000        # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from sparse_int4_gemm_amd import _lib
    return _lib.load()


def _decode(lib, **kw):
    a = dict(q=P, sq=512, o=P, so=512, lse=None, seqs=4, hq=4, hkv=2, d=128, dtype=0, k=P, v=P, pages=8, page=16, table=P,
             width=4, lens=P, max_len=64, window=0, sinks=0, scale=1.0, ws=P, wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.slim_attention_decode(*a.values())


def _prefill(lib, **kw):
    a = dict(q=P, sq=512, o=P, so=512, lse=None, tokens=9, seqs=4, hq=4, hkv=2, d=128, dtype=0, k=P, v=P, pages=8, page=16,
             table=P, width=4, lens=P, starts=P, max_len=64, window=0, sinks=0, scale=1.0, ws=P, wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.slim_attention_prefill(*a.values())


BAD = [
    (dict(dtype=2), 2), (dict(dtype=-1), 2), (dict(d=80), 2), (dict(d=0), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(page=2048), 2), (dict(hq=3), 1), (dict(hkv=0), 1), (dict(hq=0), 1), (dict(hq=2048), 1), (dict(seqs=-1), 1),
    (dict(seqs=(1 << 22) + 1), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(q=P + 8), 1), (dict(o=P + 2), 1), (dict(k=P + 4), 1),
    (dict(table=P + 2), 1), (dict(lens=P + 1), 1), (dict(lse=P + 2), 1), (dict(sq=508), 1), (dict(sq=516), 1),
    (dict(so=504), 1), (dict(sq=-512), 1), (dict(sq=1 << 40), 1), (dict(pages=0), 1), (dict(pages=1 << 25), 1),
    (dict(width=0), 1), (dict(width=1 << 27), 1), (dict(max_len=-1), 1), (dict(max_len=1 << 31), 1),
    (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(window=1 << 31), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(ws=None), 1), (dict(ws=P + 8), 1), (dict(wsb=16000), 1),
]


@pytest.mark.parametrize("kw,code", BAD)
def test_decode_rejects_bad_arguments(lib, kw, code):
    assert _decode(lib, **kw) == code
    assert lib.slim_last_error()


@pytest.mark.parametrize("kw,code", BAD + [(dict(starts=P + 2), 1), (dict(starts=None), 1), (dict(tokens=-1), 1),
                                           (dict(tokens=(1 << 22) + 1), 1), (dict(seqs=0), 1)])
def test_prefill_rejects_bad_arguments(lib, kw, code):
    assert _prefill(lib, **kw) == code
    assert lib.slim_last_error()


def test_nothing_to_do(lib):
    assert _decode(lib, seqs=0, q=None, o=None, k=None, ws=None) == 0
    assert _prefill(lib, tokens=0, q=None, o=None, k=None, ws=None) == 0
    assert lib.slim_kv_append(None, 0, None, 0, 0, 3, 2, 64, 0, None, 1, None, P, None, None, 1, 16, None) == 0
    assert lib.slim_kv_copy_pages(None, None, 1, 4, 256, None, None, 0, None) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(d=32), 2), (dict(page=24), 2), (dict(dtype=9), 2), (dict(heads=0), 1), (dict(heads=1025), 1), (dict(K=None), 1),
    (dict(V=P + 8), 1), (dict(sk=250), 1), (dict(sv=248), 1), (dict(tokens=-1), 1), (dict(seqs=0), 1), (dict(starts=None), 1),
    (dict(starts=P + 1), 1), (dict(kp=None), 1), (dict(vp=P + 4), 1), (dict(pages=0), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(width=0), 1),
])
def test_append_rejects_bad_arguments(lib, kw, code):
    a = dict(K=P, sk=256, V=P, sv=256, tokens=7, seqs=2, heads=2, d=128, dtype=0, table=P, width=4, lens=P, starts=P, kp=P,
             vp=P, pages=8, page=16, stream=None)
    a.update(kw)
    assert lib.slim_kv_append(*a.values()) == code
    assert lib.slim_last_error()


@pytest.mark.parametrize("kw", [dict(layers=0), dict(layers=5000), dict(pages=0), dict(nbytes=0), dict(nbytes=24), dict(n=-1),
                                dict(nbytes=1 << 31), dict(k=None), dict(v=P + 8), dict(src=None), dict(dst=P + 2)])
def test_copy_rejects_bad_arguments(lib, kw):
    a = dict(k=P, v=P, layers=2, pages=8, nbytes=4096, src=P, dst=P, n=3, stream=None)
    a.update(kw)
    assert lib.slim_kv_copy_pages(*a.values()) == 1
    assert lib.slim_last_error()


def test_workspace_sizes(lib):
    f = lib.slim_attention_workspace_bytes
    for args in [(1, 1, 32, 32, 128), (64, 64, 32, 8, 128), (8192, 1, 32, 8, 128), (1 << 22, 1 << 22, 1024, 1, 256),
                 (1 << 22, 1, 1024, 1024, 64), (0, 0, 1, 1, 64)]:
        n = f(*args)
        assert n >= 16384 and n % 256 == 0 and n < 1 << 30
    for args in [(-1, 1, 1, 1, 64), (1, 1, 3, 2, 64), (1, 1, 1, 1, 80), (1 << 23, 1, 1, 1, 64), (1, 1, 2048, 1, 64),
                 (1, 1, 1, 0, 64), ((1 << 63) - 1, (1 << 63) - 1, 1, 1, 64)]:
        assert f(*args) == 0


def test_binding_refuses_tensors_that_do_not_fit():
    torch = pytest.importorskip("torch")
    import sparse_int4_gemm_amd as slim
    pool = torch.empty(4, 2, 16, 64, dtype=torch.float16)
    q = torch.empty(3, 4, 64, dtype=torch.float16)
    ints = torch.zeros(3, dtype=torch.int32)
    table = torch.zeros(3, 2, dtype=torch.int32)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):                      # host tensors
        slim.attention_decode(q, pool, pool, table, ints, ws=ws, out=q)
    with pytest.raises(ValueError):
        slim.kv_append(q[:, :2], q[:, :2], pool, pool, table, ints)
    with pytest.raises(ValueError):
        slim.kv_copy_pages(pool, pool, ints, ints)
    with pytest.raises(ValueError):
        slim.attention_decode(q[0], pool, pool, table, ints, ws=ws, out=q)
    with pytest.raises(ValueError):
        slim.attention_prefill(q, pool[0], pool[0], table, ints, None, ws=ws, out=q)
    with pytest.raises(ValueError):
        slim.workspace_attention(1, 1, 3, 2, 64)

"""What KVCache refuses before it allocates or hands out anything."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("args,kw,error", [
    ((0, 4, 1, 64), {}, ValueError), ((1, 0, 1, 64), {}, ValueError), ((1, 4, 0, 64), {}, ValueError),
    ((1, 4, -1, 64), {}, ValueError), ((1, 4, 1, 0), {}, ValueError), ((1, 4, 1, 80), {}, ValueError),
    ((1, 4, 1, 512), {}, ValueError), ((1, 4, 2048, 64), {}, ValueError), ((5000, 4, 1, 64), {}, ValueError),
    ((1, (1 << 24) + 1, 1, 64), {}, ValueError), ((1, 4, 1, 64), dict(page_size=0), ValueError),
    ((1, 4, 1, 64), dict(page_size=-64), ValueError), ((1, 4, 1, 64), dict(page_size=8), ValueError),
    ((1, 4, 1, 64), dict(page_size=48), ValueError), ((1, 4, 1, 64), dict(page_size=2048), ValueError),
    ((1, 4, 1, 64), dict(dtype=torch.float32), TypeError), ((1, 4, 1, 64), dict(dtype=torch.int16), TypeError),
])
def test_the_constructor_refuses(monkeypatch, args, kw, error):
    import sparse_int4_gemm_amd as slim
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocated"))
    with pytest.raises(error):
        slim.KVCache(*args, **kw)


@pytest.mark.parametrize("page_size", [0, -4])
def test_page_sizes_that_would_never_fill(page_size):
    import sparse_int4_gemm_amd as slim
    with pytest.raises(ValueError):
        slim.KVCache(1, 4, 1, 1, page_size=page_size, dtype=torch.float32, device="cpu")

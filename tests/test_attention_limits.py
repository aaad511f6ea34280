"""The sizes that the header allows pass the checks of the C boundary, the first past them do not."""
import pytest

from test_attention_abi import P, _decode, _prefill, lib  # noqa: F401


def accepted(lib, code):
    """Every check of the arguments passed: what is left to refuse is the device."""
    return code in (2, 3) and b"evice" in lib.slim_last_error()


@pytest.fixture(autouse=True)
def without_a_device():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the pointers are none: only where no device can take the call")


@pytest.mark.parametrize("kw", [dict(hq=1024, hkv=64, d=128, sq=1024 * 128, so=1024 * 128),
                                dict(hq=1024, hkv=1, d=256, sq=1024 * 256, so=3 * 1024 * 256), dict(sq=1 << 22, so=1 << 22)])
@pytest.mark.parametrize("call", [_decode, _prefill])
def test_long_rows_pass(lib, call, kw):  # noqa: F811
    assert accepted(lib, call(lib, **kw)), lib.slim_last_error()


@pytest.mark.parametrize("kw", [dict(sq=(1 << 22) + 8), dict(so=(1 << 22) + 8), dict(hq=1024, hkv=1, d=256, sq=1 << 17, so=1 << 18)])
@pytest.mark.parametrize("call", [_decode, _prefill])
def test_longer_strides_are_refused(lib, call, kw):  # noqa: F811
    assert call(lib, **kw) == 1 and b"stride" in lib.slim_last_error()


def test_append_takes_them_too(lib):  # noqa: F811
    a = dict(K=P, sk=1 << 22, V=P, sv=1 << 18, tokens=7, seqs=2, heads=1024, d=256, dtype=0, table=P, width=4, lens=P, starts=P,
             kp=P, vp=P, pages=8, page=16, stream=None)
    assert accepted(lib, lib.slim_kv_append(*a.values())), lib.slim_last_error()
    a["sk"] += 8
    assert lib.slim_kv_append(*a.values()) == 1

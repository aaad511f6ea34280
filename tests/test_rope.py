"""Rotary positions and the 4-bit cache without a GPU: what the entry points
refuse, at the C boundary and in the binding, the frequencies against their
formulas, and the oracles against facts of their own."""
import ctypes
import math

import numpy as np
import pytest

from oracle import q4_ref, rope_ref

P = 0x10000        # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from sparse_int4_gemm_amd import _lib
    return _lib.load()


def rotation(freqs=P, rot_dim=64, interleaved=0, magnitude=1.0):
    from sparse_int4_gemm_amd import _lib
    return ctypes.byref(_lib.Rotation(freqs, rot_dim, interleaved, magnitude))


def call(f, base, kw):
    a = dict(base)
    unknown = set(kw) - set(a)
    assert not unknown, unknown
    a.update(kw)
    return f(*a.values())


ROPE = dict(x=P, sx=512, y=2 * P, sy=512, tokens=9, heads=4, d=128, dtype=0, positions=P, rot=None, stream=None)
APPEND = dict(q=P, sq=512, qo=2 * P, sqo=512, hq=4, k=P, sk=256, v=P, sv=256, tokens=9, seqs=4, hkv=2, d=128, dtype=0,
              table=P, width=4, lens=P, starts=P, kp=P, vp=P, pages=8, page=16, rot=None, stream=None)
READ = {n: x for n, x in APPEND.items() if n not in ("q", "sq", "qo", "sqo", "hq", "rot")}
DECODE = dict(q=P, sq=512, o=P, so=512, lse=None, seqs=4, hq=4, hkv=2, d=128, dtype=0, k=P, v=P, pages=8, page=16, table=P,
              width=4, lens=P, max_len=64, window=0, sinks=0, scale=1.0, ws=P, wsb=1 << 30, stream=None)
PREFILL = dict(q=P, sq=512, o=P, so=512, lse=None, tokens=9, seqs=4, hq=4, hkv=2, d=128, dtype=0, k=P, v=P, pages=8, page=16,
               table=P, width=4, lens=P, starts=P, max_len=64, window=0, sinks=0, scale=1.0, ws=P, wsb=1 << 30, stream=None)

BAD_ROTATIONS = [dict(freqs=None), dict(freqs=P + 4), dict(rot_dim=0), dict(rot_dim=-8), dict(rot_dim=12), dict(rot_dim=136),
                 dict(rot_dim=1 << 40), dict(interleaved=2), dict(interleaved=-1), dict(magnitude=float("nan")),
                 dict(magnitude=float("inf"))]


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(d=0), 2), (dict(d=12), 2), (dict(d=1032), 2), (dict(d=-8), 2), (dict(tokens=-1), 1),
    (dict(tokens=(1 << 22) + 1), 1), (dict(heads=0), 1), (dict(heads=1025), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(x=P + 8), 1), (dict(y=P + 2), 1), (dict(sx=504), 1), (dict(sx=508), 1), (dict(sy=520 - 16), 1), (dict(sx=-512), 1),
    (dict(sx=1 << 23), 1), (dict(positions=None), 1), (dict(positions=P + 2), 1), (dict(y=P, sy=520), 1)])
def test_rope_rejects_bad_arguments(lib, kw, code):
    assert call(lib.slim_rope, ROPE, dict(rot=rotation(), **kw)) == code
    assert lib.slim_last_error()


@pytest.mark.parametrize("kw", BAD_ROTATIONS)
def test_bad_rotations_are_rejected(lib, kw):
    for f, base in ((lib.slim_rope, ROPE), (lib.slim_kv_append_rope, APPEND), (lib.slim_kv_append_q4, APPEND)):
        assert call(f, base, dict(rot=rotation(**kw))) == 1
        assert lib.slim_last_error()


BAD_CACHE = [(dict(dtype=2), 2), (dict(d=80), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(page=2048), 2), (dict(hkv=0), 1),
             (dict(seqs=-1), 1), (dict(seqs=0), 1), (dict(seqs=(1 << 22) + 1), 1), (dict(tokens=-1), 1),
             (dict(tokens=(1 << 22) + 1), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(table=P + 2), 1),
             (dict(lens=P + 1), 1), (dict(starts=P + 2), 1), (dict(starts=None), 1), (dict(pages=0), 1), (dict(pages=1 << 25), 1),
             (dict(width=0), 1), (dict(width=1 << 27), 1)]
BAD_ROWS = [(dict(k=None), 1), (dict(v=None), 1), (dict(k=P + 8), 1), (dict(v=P + 2), 1), (dict(kp=None), 1), (dict(vp=None), 1),
            (dict(kp=P + 8), 1), (dict(vp=P + 4), 1), (dict(sk=248), 1), (dict(sv=252), 1), (dict(sk=-256), 1),
            (dict(sv=1 << 23), 1)]
BAD_QUERIES = [(dict(q=None), 1), (dict(qo=None), 1), (dict(hq=3), 1), (dict(hq=0), 1), (dict(hq=2048), 1), (dict(q=P + 8), 1),
               (dict(qo=P + 8), 1), (dict(sq=504), 1), (dict(sqo=508), 1), (dict(qo=P, sqo=520), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_ROWS + BAD_QUERIES)
def test_appends_reject_bad_arguments(lib, kw, code):
    for f in (lib.slim_kv_append_rope, lib.slim_kv_append_q4):
        assert call(f, APPEND, dict(rot=rotation(), **kw)) == code
        assert lib.slim_last_error()


def test_appends_need_a_rotation_where_something_turns(lib):
    assert call(lib.slim_kv_append_rope, APPEND, {}) == 1
    assert call(lib.slim_kv_append_rope, APPEND, dict(q=None, qo=None)) == 1
    assert call(lib.slim_kv_append_q4, APPEND, {}) == 1          # queries without one


@pytest.mark.parametrize("kw,code", BAD_CACHE + BAD_ROWS)
def test_read_rejects_bad_arguments(lib, kw, code):
    assert call(lib.slim_kv_read_q4, READ, kw) == code
    assert lib.slim_last_error()


BAD_ATTENTION = [
    (dict(dtype=2), 2), (dict(d=80), 2), (dict(page=8), 2), (dict(page=48), 2), (dict(hq=3), 1), (dict(hkv=0), 1),
    (dict(hq=2048), 1), (dict(seqs=-1), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(q=P + 8), 1), (dict(o=P + 2), 1), (dict(k=P + 4), 1),
    (dict(lse=P + 2), 1), (dict(sq=508), 1), (dict(so=504), 1), (dict(pages=0), 1), (dict(width=1 << 27), 1),
    (dict(max_len=-1), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(scale=float("nan")), 1), (dict(ws=None), 1),
    (dict(ws=P + 8), 1), (dict(wsb=16000), 1)]


@pytest.mark.parametrize("kw,code", BAD_ATTENTION)
def test_attention_rejects_bad_arguments(lib, kw, code):
    assert call(lib.slim_attention_decode_q4, DECODE, kw) == code and lib.slim_last_error()
    assert call(lib.slim_attention_prefill_q4, PREFILL, kw) == code and lib.slim_last_error()


def test_nothing_to_do(lib):
    assert call(lib.slim_rope, ROPE, dict(rot=rotation(), tokens=0, x=None, y=None, positions=None)) == 0
    for f in (lib.slim_kv_append_rope, lib.slim_kv_append_q4):
        assert call(f, APPEND, dict(rot=rotation(), tokens=0, q=None, qo=None, k=None, v=None, kp=None, vp=None)) == 0
    assert call(lib.slim_kv_read_q4, READ, dict(tokens=0, k=None, v=None, kp=None)) == 0
    assert call(lib.slim_attention_decode_q4, DECODE, dict(seqs=0, q=None, o=None, k=None, ws=None)) == 0
    assert call(lib.slim_attention_prefill_q4, PREFILL, dict(tokens=0, q=None, o=None, k=None, ws=None)) == 0


def test_page_bytes(lib):
    assert lib.slim_q4_page_bytes(8, 64, 128) == 8 * 64 * 68
    assert lib.slim_q4_page_bytes(1, 16, 96) == 816
    for bad in ((0, 64, 128), (-1, 64, 128), (1025, 64, 128), (8, 63, 128), (8, 2048, 128), (8, 64, 80), (8, 64, -128)):
        assert lib.slim_q4_page_bytes(*bad) == 0
    for heads in (1, 3, 1024):
        for page in (16, 64, 1024):
            for dim in (64, 96, 128, 256):
                assert lib.slim_q4_page_bytes(heads, page, dim) % 16 == 0


# ------------------------------------------------------------- the binding
def test_frequencies():
    from sparse_int4_gemm_amd import rope_frequencies
    for rot, base in ((8, 10000.0), (64, 10000.0), (128, 500000.0)):
        plain = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
        f, m = rope_frequencies(rot, base)
        assert np.allclose(f.numpy(), plain, rtol=1e-14) and m == 1.0
        f, m = rope_frequencies(rot, base, "linear", 4.0)
        assert np.allclose(f.numpy(), plain / 4.0, rtol=1e-14) and m == 1.0
        f, m = rope_frequencies(rot, base, "ntk", 4.0)
        assert f[0] == 1.0 and np.isclose(f[-1], plain[-1] / 4.0, rtol=1e-13) and m == 1.0
        f, m = rope_frequencies(rot, base, "yarn", 4.0, 4096)
        turns = 4096 * plain / (2 * math.pi)
        assert np.allclose(m, 0.1 * math.log(4.0) + 1.0)
        assert np.allclose(f.numpy()[turns >= 32 * 1.4], plain[turns >= 32 * 1.4], rtol=1e-14) or rot == 8
        assert np.allclose(f.numpy()[turns <= 0.6], plain[turns <= 0.6] / 4.0, rtol=1e-14)
        assert (f.numpy() <= plain).all() and (f.numpy() >= plain / 4.0 * (1 - 1e-14)).all() and (np.diff(f.numpy()) < 0).all()


def test_rotations_that_cannot_be_made():
    import torch
    from sparse_int4_gemm_amd import Rope, rope_frequencies
    for bad in (dict(rot_dim=0), dict(rot_dim=12), dict(rot_dim=64, base=1.0), dict(rot_dim=64, base=float("nan")),
                dict(rot_dim=64, scaling="other"), dict(rot_dim=64, scaling="linear", factor=0.5),
                dict(rot_dim=64, scaling="yarn", factor=2.0), dict(rot_dim=64, scaling="yarn", original_len=4096, turns=(1.0, 32.0))):
        with pytest.raises(ValueError):
            rope_frequencies(**bad)
        with pytest.raises(ValueError):
            Rope(**bad, device="cpu")
    with pytest.raises(ValueError):
        Rope(64, freqs=torch.zeros(32), device="cpu")                  # not float64
    with pytest.raises(ValueError):
        Rope(64, freqs=torch.zeros(64, dtype=torch.float64), device="cpu")
    with pytest.raises(ValueError):
        Rope(64, magnitude=float("inf"), device="cpu")
    own = torch.linspace(0, 1, 32, dtype=torch.float64)
    r = Rope(64, freqs=own, interleaved=True, magnitude=0.5, device="cpu")
    assert torch.equal(r.freqs, own) and r.magnitude == 0.5 and r.params.interleaved == 1 and r.params.rot_dim == 64


def test_cache_of_four_bits_on_the_host():
    from sparse_int4_gemm_amd import KVCache
    import torch
    c = KVCache(2, 8, 3, 96, page_size=16, device="cpu", bits=4)
    assert c.k.dtype == torch.uint8 and c.k.shape == (2, 8, 3, 16, 51) and c.v.shape == c.k.shape and c.bits == 4
    s = c.add()
    assert c.extend([s], [40]).max_len == 40 and c.free_pages == 5
    for bits in (0, 8, 3, "4"):
        with pytest.raises(ValueError):
            KVCache(1, 8, 1, 128, device="cpu", bits=bits)
    with pytest.raises(ValueError):
        KVCache(1, 8, 1, 80, device="cpu", bits=4)                     # no whole groups of 32
    with pytest.raises(ValueError):
        KVCache(1, 8, 1, 128, page_size=8, device="cpu", bits=4)


# -------------------------------------------------------------- the oracles
def test_the_rotation_keeps_lengths_and_differences_of_positions():
    rng = np.random.default_rng(1)
    f = np.array([1.0, 0.3, 0.01, 1e-4])
    q, k = rng.standard_normal((2, 3, 1, 12))
    for inter in (False, True):
        a = rope_ref.turn(q, [5, 6, 7], f, inter)
        assert np.allclose((a ** 2).sum(-1), (q ** 2).sum(-1)) and np.array_equal(a[..., 8:], q[..., 8:])
        b, c = rope_ref.turn(k, [2, 3, 4], f, inter), rope_ref.turn(k, [102, 103, 104], f, inter)
        assert np.allclose((a * b).sum(-1), (rope_ref.turn(q, [105, 106, 107], f, inter) * c).sum(-1))
        assert np.allclose(rope_ref.turn(a, [-5, -6, -7], f, inter), q)
    assert np.allclose(rope_ref.turn([[[1.0, 0.0]]], [1], [math.pi / 2]), [[[0.0, 1.0]]])


def test_codes_of_known_values():
    x = np.zeros(32)
    x[:16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.26, 0.74, 0.76, 5.01, 7, -5]
    code, e = q4_ref.encode(x, "fp16")
    assert e[0] == 127
    assert code[:16].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 9, 1, 2, 7, 7, 14]
    for top, want in ((7.0, 0), (7.0 + 2.0 ** -20, 1), (3.5, -1), (2.0 ** -40, -23), (0.0, -23), (65504.0, 13), (1e5, 13)):
        assert int(q4_ref.encode(np.full(32, top), "fp16")[1][0]) - 127 == want
    assert int(q4_ref.encode(np.full(32, 3.3e38), "bf16")[1][0]) - 127 == 125
    for bad in (np.inf, -np.inf, np.nan):
        x[3] = bad
        code, e = q4_ref.encode(x, "bf16")
        assert e[0] == 255 and not code.any() and np.isnan(q4_ref.decode(code, e)).all()


def test_no_element_moves_by_more_than_its_half_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((500, 64)) * 2.0 ** rng.integers(-9, 9, (500, 1))
    code, e = q4_ref.encode(x, "fp16")
    by = np.repeat(2.0 ** (e.astype(np.float64) - 127), 32, -1)
    assert (np.abs(q4_ref.decode(code, e) - x) <= by).all() and (np.abs(x) <= 7 * by).all()
    pool, scale = code.reshape(1, 5, 100, 64)[:, :, :96], e.reshape(1, 5, 100, 2)[:, :, :96]
    back = q4_ref.unpack(q4_ref.pack(pool, scale))
    assert np.array_equal(back[0], pool) and np.array_equal(back[1], scale)

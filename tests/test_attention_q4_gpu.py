"""slim_attention_decode_q4 and slim_attention_prefill_q4 against the fp64
oracle on the values that the codes stand for (each exact in the type, so the
bound of the 16-bit calls holds): types, head layouts, head sizes, page sizes,
lengths from none to several splits, windows and sinks, rows that see nothing,
whatever lies in places that are not seen, strides, streams, graphs."""
import numpy as np
import pytest

from attention_helpers import bound, check, host, reference
from q4_helpers import junk_rows, q4_case, scale_byte

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import sparse_int4_gemm_amd as slim
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    slim._lib.load()
    return torch, slim


def run(env, c, window=0, sinks=0, lse=False, **kw):
    torch, slim = env
    kw.setdefault("out", torch.full_like(c["q"], 77.0))
    if lse:
        kw["lse"] = torch.full((c["q"].shape[0], c["q"].shape[1]), 77.0, device="cuda")
    args = (c["q"], c["k4"], c["v4"], c["d_table"], c["d_lens"])
    kw = dict(window=window, sinks=sinks, scale=c["scale"], **kw)
    if c["starts"] is None:
        y = slim.attention_decode_q4(*args, **kw)
    else:
        y = slim.attention_prefill_q4(*args, c["d_starts"], **kw)
    torch.cuda.synchronize()
    return (y, kw["lse"]) if lse else y


HEADS = [(1, 1), (8, 2), (14, 2), (16, 1), (20, 1), (40, 1)]
DTYPES = ["fp16", "bf16"]
WINDOWS = [(1, 0), (1, 1), (7, 3), (64, 4), (100, 200), (1000, 16), (1 << 30, 5), (33, 1 << 30)]


# ------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", HEADS)
def test_decode_head_layouts(env, dtype, dim, q_heads, kv_heads):
    c = q4_case(env[0], 1, dtype, [1, 2, 31, 33, 64, 100, 300], q_heads, kv_heads, dim, 16)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
@pytest.mark.parametrize("dtype,dim", [("fp16", 128), ("bf16", 96)])
def test_decode_page_sizes_and_lengths(env, dtype, dim, page):
    c = q4_case(env[0], 2, dtype, [0, 1, 15, 16, 17, 63, 65, 127, 128, 129, 1000, 1023, 1024, 1025], 4, 2, dim, page)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("lens", [[5000], [4097, 1], [8191, 3, 0, 8191]])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(2, 2, 128), (8, 1, 64), (3, 1, 96), (2, 1, 256)])
def test_decode_long_axis_is_split_and_joined(env, lens, q_heads, kv_heads, dim):
    c = q4_case(env[0], 3, "fp16", lens, q_heads, kv_heads, dim, 64)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    for max_len in (0, 1, 100, 1 << 30):
        check(c, run(env, c, max_len=max_len), what=f"max_len={max_len}")


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("page", [16, 128])
def test_decode_window_and_sinks(env, page, window, sinks):
    c = q4_case(env[0], 4, "bf16", [1, 5, 64, 99, 101, 300, 1500, 4000], 4, 1, 64, page)
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("most", [200, 900])
def test_decode_many_sequences(env, most):
    """More than a round of workgroups; from 512 keys on the longest go first."""
    rng = np.random.default_rng(5)
    c = q4_case(env[0], 5, "fp16", [int(n) for n in rng.integers(0, most, 300)], 4, 4, 64, 32)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


def test_decode_peaked_and_large_scores(env):
    c = q4_case(env[0], 6, "fp16", [700, 64, 1], 4, 2, 128, 16, q_std=3.0)
    check(c, run(env, c))
    c["scale"] = -c["scale"]
    check(c, run(env, c), what="negative scale")
    c["scale"] = 0.0
    check(c, run(env, c), what="scale 0: the mean of the values")


# ------------------------------------------------------ prompts and chunks
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", HEADS)
def test_prefill_head_layouts(env, dtype, dim, q_heads, kv_heads):
    c = q4_case(env[0], 11, dtype, [1, 40, 130], q_heads, kv_heads, dim, 16, new=[1, 33, 70])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("dtype,dim", [("fp16", 128), ("bf16", 128), ("fp16", 96), ("bf16", 256), ("bf16", 64)])
def test_prefill_lengths_and_prefixes(env, dtype, dim, page):
    new = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 257]
    pre = [5, 0, 100, 1, 0, 64, 300, 17, 0, 128, 31, 0]
    c = q4_case(env[0], 12, dtype, [n + p for n, p in zip(new, pre)], 2, 1, dim, page, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_window_and_sinks(env, dim, window, sinks):
    c = q4_case(env[0], 13, "fp16", [300, 1, 500, 700], 4, 2, dim, 16, new=[300, 1, 20, 260])
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("new,pre", [([3], [6000]), ([17, 1], [4000, 9000]), ([1, 1, 1], [10, 5000, 0])])
@pytest.mark.parametrize("q_heads,kv_heads", [(2, 2), (8, 1)])
def test_prefill_few_rows_on_a_long_prefix(env, new, pre, q_heads, kv_heads):
    c = q4_case(env[0], 14, "bf16", [n + p for n, p in zip(new, pre)], q_heads, kv_heads, 128, 64, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    check(c, run(env, c, window=1000, sinks=4), window=1000, sinks=4)
    for max_len in (0, 1, 1 << 30):
        check(c, run(env, c, max_len=max_len), what=f"max_len={max_len}")


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("fp16", 128), ("bf16", 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5), (500, 0)])
def test_prefill_more_row_blocks_than_a_round_of_workgroups(env, dtype, dim, window, sinks):
    """Many short sequences with one behind a prefix of more than 64 tiles, unsplit: pages are looked up again on the way."""
    new = [3] + [int(n) for n in np.random.default_rng(71).integers(0, 9, 70)]
    pre = [9000] + [int(n) for n in np.random.default_rng(72).integers(0, 150, 70)]
    c = q4_case(env[0], 71, dtype, [n + p for n, p in zip(new, pre)], 8, 4, dim, 32, new=new)
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_long_unsplit_walk_of_both_wave_groups(env, dim):
    new = [2] + [1] * 45
    pre = [9500] + [int(n) for n in np.random.default_rng(73).integers(0, 200, 45)]
    c = q4_case(env[0], 73, "fp16", [n + p for n, p in zip(new, pre)], 4, 4, dim, 16, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("q_heads,kv_heads,new,pre", [(12, 4, 700, 0), (4, 4, 600, 333), (64, 8, 130, 40), (7, 7, 129, 1)])
def test_prefill_row_blocks_cross_tokens_and_heads(env, q_heads, kv_heads, new, pre):
    c = q4_case(env[0], 74, "bf16", [new + pre, 5], q_heads, kv_heads, 64, 64, new=[new, 2])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


def test_prefill_without_starts_is_decode(env):
    torch, slim = env
    c = q4_case(torch, 18, "fp16", [0, 1, 64, 1000], 8, 2, 128, 32)
    y = slim.attention_prefill_q4(c["q"], c["k4"], c["v4"], c["d_table"], c["d_lens"], None, scale=c["scale"])
    check(c, y)


# -------------------------------------------------- places that are not seen
@pytest.mark.parametrize("junk", ["any", "nan", "max"])
@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("dtype,dim", [("fp16", 128), ("bf16", 96), ("bf16", 64), ("fp16", 256)])
def test_unseen_places_do_not_reach_a_row(env, form, dtype, dim, junk):
    """Pages nobody owns, the tails of last pages and keys outside the window hold any bytes, NaN scales, or scales whose
    values pass the type's range."""
    torch, slim = env
    new = None if form == "decode" else [70, 1, 33, 200]
    c = q4_case(torch, 21, dtype, [70, 9, 333, 200], 4, 2, dim, 16, new=new)
    scale = {"any": None, "nan": 255, "max": 254}[junk]
    rng = np.random.default_rng(21)
    owned = {}
    for b in range(4):
        for j in range(int(c["lens"][b])):
            owned.setdefault(int(c["table"][b, j // 16]), set()).add(j % 16)
    for p in range(c["k"].shape[0]):
        for pool in ("k4", "v4"):
            junk_rows(torch, c[pool], p, [r for r in range(16) if r not in owned.get(p, ())], rng, scale)
    check(c, run(env, c), what="unowned places")
    window, sinks = 40, 2
    first = (333 - (1 if new is None else 33)) - window + 1
    for j in range(sinks, first):
        for pool in ("k4", "v4"):
            junk_rows(torch, c[pool], int(c["table"][2, j // 16]), [j % 16], rng, scale)
    check(c, run(env, c, window, sinks), window=window, sinks=sinks, what="outside the window")


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 128), ("fp16", 96), ("bf16", 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_prefill_later_nan_keys_do_not_reach_earlier_rows(env, dtype, dim, window, sinks):
    """A NaN group of a key and value that only some rows of a tile see: the others are as if it were clean."""
    torch, slim = env
    c = q4_case(torch, 22, dtype, [150], 2, 1, dim, 16, new=[150])
    at = (5, 40, 77, 100, 149)
    clean, _, mass = reference(c, window, sinks)
    for j in at:
        for pool in ("k4", "v4"):
            scale_byte(c[pool], int(c["table"][0, j // 16]), 0, j % 16, 1).fill_(255)
    got = host(run(env, c, window, sinks))
    for i in range(150):
        if any(j <= i and (not window or j > i - window or j < sinks) for j in at):
            continue
        over = np.abs(got[i] - clean[i]) - bound(c, clean[i], mass[i])
        assert over.max() <= 0, f"row {i}: {over.max()}"
    assert np.isnan(got[149]).all()


@pytest.mark.parametrize("dtype,dim,heads", [("fp16", 64, 2), ("bf16", 128, 20), ("fp16", 96, 1), ("bf16", 256, 3)])
@pytest.mark.parametrize("lens", [[50, 90], [5200, 50]])
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_a_seen_nan_group_of_a_value_reaches_only_its_elements(env, form, dtype, dim, heads, lens):
    torch, slim = env
    c = q4_case(torch, 23, dtype, lens, heads, 1, dim, 16, new=None if form == "decode" else [1, 40])
    want, _, mass = reference(c)
    scale_byte(c["v4"], int(c["table"][0, 0]), 0, 3, 1).fill_(255)
    got = host(run(env, c))
    bad = np.zeros(got.shape, dtype=bool)
    bad[0, :, 32:64] = True
    assert np.array_equal(np.isnan(got), bad)
    assert ((np.abs(got - want) - bound(c, want, mass))[~bad] <= 0).all()


def test_bad_table_entries_hold_no_keys(env):
    torch, slim = env
    for new in (None, [33, 64, 20]):
        c = q4_case(torch, 24, "fp16", [200, 64, 333], 4, 2, 128, 16, new=new)
        for b, i, x in [(0, 3, -1), (0, 12, 10 ** 6), (2, 0, -2 ** 31), (2, 20, 2 ** 31 - 1), (1, 0, -5), (1, 1, -5),
                        (1, 2, -5), (1, 3, c["k"].shape[0])]:
            c["table"][b, i] = x
        c["d_table"].copy_(torch.from_numpy(c["table"]))
        y, lse = run(env, c, lse=True)
        check(c, y, lse)


def test_lengths_past_the_table_and_negative_lengths(env):
    torch, slim = env
    for new in (None, [2, 5, 3, 1]):
        c = q4_case(torch, 25, "fp16", [64, 48, 64, 30], 2, 2, 64, 16, new=new)
        c["lens"] = np.asarray([500, -3, 2 ** 20, 30], dtype=np.int32)
        c["d_lens"].copy_(torch.from_numpy(c["lens"]))
        y, lse = run(env, c, lse=True)
        check(c, y, lse)


def test_rows_of_no_sequence_are_left_alone(env):
    torch, slim = env
    c = q4_case(torch, 27, "fp16", [40, 70], 4, 2, 64, 16, new=[40, 7])
    want = run(env, c)
    q = torch.cat([c["q"][:9], c["q"], torch.randn(83, 4, 64, device="cuda").half()])
    out = torch.full_like(q, 77.0)
    slim.attention_prefill_q4(q, c["k4"], c["v4"], c["d_table"], c["d_lens"], c["d_starts"] + 9, scale=c["scale"], out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[9:56], want) and (out[56:] == 77).all() and (out[:9] == 77).all()


# ----------------------------------------------------- strides, streams, graphs
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_strided_rows(env, form):
    torch, slim = env
    c = q4_case(torch, 31, "bf16", [33, 100, 64], 4, 2, 96, 16, new=None if form == "decode" else [33, 5, 64])
    want = run(env, c)
    tokens = c["q"].shape[0]
    joint = torch.randn(tokens, 8, 96, device="cuda").bfloat16()
    joint[:, 2:6] = c["q"]
    wide = torch.full((tokens, 7, 96), 77.0, device="cuda", dtype=torch.bfloat16)
    got = run(env, dict(c, q=joint[:, 2:6]), out=wide[:, 1:5])
    assert torch.equal(got, want) and (wide[:, :1] == 77).all() and (wide[:, 5:] == 77).all()


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_repeats_bit_for_bit_on_one_workspace_and_other_streams(env, form):
    torch, slim = env
    ws = slim.workspace_attention(400, 400, 8, 4, 256)
    first = {}
    side = torch.cuda.Stream()
    for turn in range(3):
        for i, (lens, new) in enumerate([([3000, 10], [1, 3]), ([5], [5]), ([100] * 40, [7] * 40)]):
            c = q4_case(torch, 40 + i, "fp16", lens, 4, 2, 128, 64, new=None if form == "decode" else new)
            y = run(env, c, ws=ws).clone()
            first.setdefault(i, y)
            assert torch.equal(y, first[i])
            y = torch.empty_like(c["q"])
            torch.cuda.synchronize()
            z = run(env, c, out=y, stream=side)
            side.synchronize()
            assert torch.equal(z, first[i])


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_graph_replays_follow_the_device_arrays(env, form):
    torch, slim = env
    new = None if form == "decode" else [3, 20]
    cs = [q4_case(torch, 50 + i, "fp16", lens, 4, 2, 128, 16, new=new, width=80, pages=200)
          for i, lens in enumerate([[40, 700], [1000, 41], [20, 1280], [3, 20]])]
    names = ("q", "k4", "v4", "d_table", "d_lens")
    st = {n: cs[0][n].clone() for n in names}
    st.update(scale=cs[0]["scale"], starts=cs[0]["starts"], d_starts=cs[0]["d_starts"])
    ws = slim.workspace_attention(st["q"].shape[0], 2, 4, 2, 128)
    out = torch.empty_like(st["q"])
    run(env, st, ws=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        args = (st["q"], st["k4"], st["v4"], st["d_table"], st["d_lens"])
        if new is None:
            slim.attention_decode_q4(*args, scale=st["scale"], ws=ws, out=out)
        else:
            slim.attention_prefill_q4(*args, st["d_starts"], scale=st["scale"], ws=ws, out=out)
    for turn in range(2):
        for c in cs:
            for n in names:
                st[n].copy_(c[n])
            out.fill_(77.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            check(c, out, what=f"replay {turn}")
            assert torch.equal(out, run(env, c, ws=ws)), "replay differs from the eager call"


def test_a_run_of_them_together(env):
    """Prompts, then single tokens: turned and appended to 4 bits in one call, attended, against the 16-bit calls on the
    cache's own values."""
    torch, slim = env
    rope = slim.Rope(128, scaling="yarn", factor=4.0, original_len=64)
    cache = slim.KVCache(1, 60, 2, 128, page_size=16, bits=4)
    plain = slim.KVCache(1, 60, 2, 128, page_size=16)
    seqs = [cache.add() for _ in range(3)]
    for s in seqs:
        assert plain.add() == s
    gen = torch.Generator(device="cuda").manual_seed(5)
    for counts in ([70, 1, 33], [1, 1, 1], [1, 1, 1], [5, 0, 1]):
        batch, same = cache.extend(seqs, counts), plain.extend(seqs, counts)
        q, k, v = (torch.randn((batch.tokens, h, 128), generator=gen, device="cuda").half() for h in (8, 2, 2))
        turned = slim.kv_append_q4(k, v, cache.k[0], cache.v[0], batch.table, batch.lens, starts=batch.starts, rope=rope, q=q)
        kr, vr = slim.kv_read_q4(cache.k[0], cache.v[0], batch.table, batch.lens, starts=batch.starts, tokens=batch.tokens)
        slim.kv_append(kr, vr, plain.k[0], plain.v[0], same.table, same.lens, same.starts)
        if all(n == 1 for n in counts):
            y = slim.attention_decode_q4(turned, cache.k[0], cache.v[0], batch.table, batch.lens)
        else:
            y = slim.attention_prefill_q4(turned, cache.k[0], cache.v[0], batch.table, batch.lens, batch.starts)
        torch.cuda.synchronize()
        c = dict(q=turned, k=plain.k[0], v=plain.v[0], table=same.table.cpu().numpy(), lens=same.lens.cpu().numpy(),
                 starts=same.starts.cpu().numpy(), dtype="fp16", scale=128 ** -0.5)
        owned = sorted({p for s in seqs for p in plain.pages(s)})
        k, v = np.zeros(plain.k[0].shape), np.zeros(plain.k[0].shape)
        for p in owned:
            k[p], v[p] = np.nan_to_num(host(plain.k[0, p])), np.nan_to_num(host(plain.v[0, p]))
        check(c, y, k=k, v=v)


def test_refusals_in_the_binding(env):
    torch, slim = env
    c = q4_case(torch, 4, "fp16", [5, 9], 4, 2, 64, 16)
    good = dict(q=c["q"], kpool=c["k4"], vpool=c["v4"], table=c["d_table"], lens=c["d_lens"])
    for bad in (dict(q=c["q"].float()), dict(kpool=c["k"], vpool=c["v"]), dict(kpool=c["k4"][..., :17]), dict(q=c["q"][:, :3]),
                dict(q=c["q"][..., :32]), dict(table=c["d_table"][:1]), dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
                dict(window=-1), dict(scale=float("nan")), dict(out=c["q"][:1])):
        for f, more in ((slim.attention_decode_q4, {}), (slim.attention_prefill_q4, dict(starts=None))):
            with pytest.raises((TypeError, ValueError, slim.SlimError)):
                f(**{**good, **more, **bad})

"""slim_attention_decode and slim_attention_prefill against the fp64 oracle:
types, head layouts, head sizes, page sizes, lengths from none to several
splits, windows and sinks, rows that see nothing, whatever lies in places that
are not seen, strides, streams, graphs and repeats."""
import numpy as np
import pytest

from attention_helpers import bound, case, check, host, reference

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
    out = torch.full_like(c["q"], 77.0)
    kw.setdefault("out", out)
    if lse:
        kw["lse"] = torch.full((c["q"].shape[0], c["q"].shape[1]), 77.0, device="cuda")
    args = (c["q"], c["k"], c["v"], c["d_table"], c["d_lens"])
    kw = dict(window=window, sinks=sinks, scale=c["scale"], **kw)
    if c["starts"] is None:
        y = slim.attention_decode(*args, **kw)
    else:
        y = slim.attention_prefill(*args, c["d_starts"], **kw)
    torch.cuda.synchronize()
    return (y, kw["lse"]) if lse else y


HEADS = [(1, 1), (4, 4), (8, 2), (14, 2), (16, 1), (20, 1), (40, 1)]


# ------------------------------------------------------------- single tokens
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", HEADS)
def test_decode_head_layouts(env, dtype, dim, q_heads, kv_heads):
    c = case(env[0], 1, dtype, [1, 2, 31, 33, 64, 100, 300], q_heads, kv_heads, dim, 16)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("page", [16, 32, 64, 256, 1024])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode_page_sizes_and_lengths(env, dtype, page):
    c = case(env[0], 2, dtype, [0, 1, 15, 16, 17, 63, 65, 127, 128, 129, 1000, 1023, 1024, 1025], 4, 2, 128, page)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("lens", [[5000], [4097, 1], [8191, 3, 0, 8191]])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(2, 2, 128), (8, 1, 64), (3, 1, 96), (2, 1, 256)])
def test_decode_long_axis_is_split_and_joined(env, lens, q_heads, kv_heads, dim):
    c = case(env[0], 3, "fp16", lens, q_heads, kv_heads, dim, 64)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    # The expected length only plans the split.
    for max_len in (0, 1, 100, 1 << 30):
        check(c, run(env, c, max_len=max_len), what=f"max_len={max_len}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (100, 200), (1000, 16), (1 << 30, 5), (33, 1 << 30)])
@pytest.mark.parametrize("page", [16, 128])
def test_decode_window_and_sinks(env, page, window, sinks):
    c = case(env[0], 4, "bf16", [1, 5, 64, 99, 101, 300, 1500, 4000], 4, 1, 64, page)
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


def test_decode_many_sequences(env):
    rng = np.random.default_rng(5)
    c = case(env[0], 5, "fp16", [int(n) for n in rng.integers(0, 200, 300)], 4, 4, 64, 32)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


def test_decode_peaked_and_large_scores(env):
    c = case(env[0], 6, "fp16", [700, 64, 1], 4, 2, 128, 16, q_std=3.0)
    check(c, run(env, c))
    c["scale"] = -c["scale"]
    check(c, run(env, c), what="negative scale")
    c["scale"] = 0.0
    check(c, run(env, c), what="scale 0: the mean of the values")


# ------------------------------------------------------ prompts and chunks
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", HEADS)
def test_prefill_head_layouts(env, dtype, dim, q_heads, kv_heads):
    c = case(env[0], 11, dtype, [1, 40, 130], q_heads, kv_heads, dim, 16, new=[1, 33, 70])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prefill_lengths_and_prefixes(env, dtype, page):
    new = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 129, 257]
    pre = [5, 0, 100, 1, 0, 64, 300, 17, 0, 128, 31, 0]
    c = case(env[0], 12, dtype, [n + p for n, p in zip(new, pre)], 2, 1, 128, page, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 3), (64, 4), (100, 200), (300, 16), (1 << 30, 5), (33, 1 << 30)])
@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_window_and_sinks(env, dim, window, sinks):
    c = case(env[0], 13, "fp16", [300, 1, 500, 700], 4, 2, dim, 16, new=[300, 1, 20, 260])
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("new,pre", [([3], [6000]), ([17, 1], [4000, 9000]), ([1, 1, 1], [10, 5000, 0])])
@pytest.mark.parametrize("q_heads,kv_heads", [(2, 2), (8, 1)])
def test_prefill_few_rows_on_a_long_prefix(env, new, pre, q_heads, kv_heads):
    c = case(env[0], 14, "bf16", [n + p for n, p in zip(new, pre)], q_heads, kv_heads, 128, 64, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    check(c, run(env, c, window=1000, sinks=4), window=1000, sinks=4)
    for max_len in (0, 1, 1 << 30):
        check(c, run(env, c, max_len=max_len), what=f"max_len={max_len}")


def test_prefill_long_prompt(env):
    c = case(env[0], 15, "fp16", [1500], 2, 1, 128, 64, new=[1500])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


def test_prefill_many_sequences(env):
    rng = np.random.default_rng(16)
    new = [int(n) for n in rng.integers(0, 40, 150)]
    c = case(env[0], 16, "fp16", [n + int(p) for n, p in zip(new, rng.integers(0, 100, 150))], 2, 2, 64, 16, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


def test_prefill_peaked_scores(env):
    c = case(env[0], 17, "fp16", [200, 64], 4, 2, 128, 16, new=[200, 10], q_std=3.0)
    check(c, run(env, c))
    c["scale"] = -c["scale"]
    check(c, run(env, c), what="negative scale")


def test_prefill_without_starts_is_decode(env):
    torch, slim = env
    c = case(torch, 18, "fp16", [0, 1, 64, 1000], 8, 2, 128, 32)
    y = slim.attention_prefill(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"], None, scale=c["scale"])
    check(c, y)


# -------------------------------------------------- places that are not seen
@pytest.mark.parametrize("junk", ["nan", "inf", "-inf", "max"])
@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_unseen_places_do_not_reach_a_row(env, form, dtype, junk):
    """Pages nobody owns, the tails of last pages, keys outside the window and
    (prefill) keys that are later than a row's position: each row is compared with the
    oracle on the clean pools."""
    torch, slim = env
    new = None if form == "decode" else [70, 1, 33, 200]
    c = case(torch, 21, dtype, [70, 9, 333, 200], 4, 2, 128, 16, new=new)
    k, v = host(c["k"]), host(c["v"])
    bad = torch.finfo(c["k"].dtype).max if junk == "max" else float(junk)
    owned = {}
    for b in range(4):
        for j in range(int(c["lens"][b])):
            owned.setdefault(int(c["table"][b, j // 16]), set()).add(j % 16)
    for p in range(c["k"].shape[0]):
        for r in range(16):
            if r not in owned.get(p, ()):
                c["k"][p, :, r] = bad
                c["v"][p, :, r] = bad
    check(c, run(env, c), k=k, v=v, what="unowned places")
    # Outside the window of every row (sequence 2: positions from 300 on for prefill, 332 for decode).
    window, sinks = 40, 2
    first = (333 - (1 if new is None else 33)) - window + 1
    for j in range(sinks, first):
        c["k"][int(c["table"][2, j // 16]), :, j % 16] = bad
        c["v"][int(c["table"][2, j // 16]), :, j % 16] = bad
    check(c, run(env, c, window, sinks), window=window, sinks=sinks, k=k, v=v, what="outside the window")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("junk", ["nan", "inf"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_prefill_later_keys_do_not_reach_earlier_rows(env, dtype, junk, window, sinks):
    """A key and value that only some rows of a tile see: the others are as if it were clean."""
    torch, slim = env
    c = case(torch, 22, dtype, [150], 2, 1, 64, 16, new=[150])
    at = (5, 40, 77, 100, 149)
    clean_out, _, mass = reference(c, window, sinks)
    for j in at:
        c["k"][int(c["table"][0, j // 16]), :, j % 16] = float(junk)
        c["v"][int(c["table"][0, j // 16]), :, j % 16] = float(junk)
    got = host(run(env, c, window, sinks))
    for i in range(150):
        sees = any(j <= i and (not window or j > i - window or j < sinks) for j in at)
        if sees:
            continue
        over = np.abs(got[i] - clean_out[i]) - bound(c, clean_out[i], mass[i])
        assert over.max() <= 0, f"row {i}: {over.max()}"
    if junk == "nan":
        assert np.isnan(got[149]).all()


def test_seen_nan_value_reaches_only_its_element(env):
    torch, slim = env
    for new in (None, [50]):
        c = case(torch, 23, "fp16", [50], 2, 2, 64, 16, new=new)
        k, v = host(c["k"]), host(c["v"])
        c["v"][int(c["table"][0, 0]), 0, 3, 7] = float("nan")
        got = host(run(env, c))
        want, _, mass = reference(c, k=k, v=v)
        last = got[-1]
        assert np.isnan(last[0, 7]) and np.isfinite(np.delete(last[0], 7)).all() and np.isfinite(last[1]).all()
        assert (np.abs(last - want[-1]) - bound(c, want[-1], mass[-1]))[1].max() <= 0


def test_bad_table_entries_hold_no_keys(env):
    torch, slim = env
    for new in (None, [33, 64, 20]):
        c = case(torch, 24, "fp16", [200, 64, 333], 4, 2, 128, 16, new=new)
        for b, i, x in [(0, 3, -1), (0, 12, 10 ** 6), (2, 0, -2 ** 31), (2, 20, 2 ** 31 - 1), (1, 0, -5), (1, 1, -5),
                        (1, 2, -5), (1, 3, c["k"].shape[0])]:
            c["table"][b, i] = x
        c["d_table"].copy_(torch.from_numpy(c["table"]))
        y, lse = run(env, c, lse=True)
        check(c, y, lse)


def test_lengths_past_the_table_and_negative_lengths(env):
    torch, slim = env
    for new in (None, [2, 5, 3, 1]):
        c = case(torch, 25, "fp16", [64, 48, 64, 30], 2, 2, 64, 16, new=new)
        c["lens"] = np.asarray([500, -3, 2 ** 20, 30], dtype=np.int32)
        c["d_lens"].copy_(torch.from_numpy(c["lens"]))
        y, lse = run(env, c, lse=True)
        check(c, y, lse)


def test_more_new_tokens_than_length(env):
    """Rows at negative positions see nothing."""
    c = case(env[0], 26, "fp16", [5, 40], 2, 1, 64, 16, new=[9, 40])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    assert (host(y)[:4] == 0).all() and np.isneginf(host(lse)[:4]).all()


def test_prefill_rows_past_the_batch_are_left_alone(env):
    torch, slim = env
    c = case(torch, 27, "fp16", [40, 70], 4, 2, 64, 16, new=[40, 7])
    want = run(env, c)
    q = torch.cat([c["q"], torch.randn(83, 4, 64, device="cuda").half()])
    out = torch.full_like(q, 77.0)
    slim.attention_prefill(q, c["k"], c["v"], c["d_table"], c["d_lens"], c["d_starts"], scale=c["scale"], out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:47], want) and (out[47:] == 77).all()


def test_starts_out_of_range_stay_in_range(env):
    """Broken starts: rows that exist are computed or left alone, none outside is touched."""
    torch, slim = env
    c = case(torch, 28, "fp16", [40, 70], 4, 2, 64, 16, new=[40, 7])
    for s in ([-5, 40, 10 ** 6], [0, 2 ** 31 - 1, 3], [30, 20, 10], [10 ** 6, 10 ** 6, 10 ** 6], [-2 ** 31, 0, 2 ** 31 - 1]):
        buf = torch.full((47 + 256, 4, 64), 77.0, device="cuda", dtype=torch.float16)
        slim.attention_prefill(c["q"], c["k"], c["v"], c["d_table"], c["d_lens"],
                               torch.tensor(s, dtype=torch.int32, device="cuda"), scale=c["scale"], out=buf[128:175])
        torch.cuda.synchronize()
        assert (buf[:128] == 77).all() and (buf[175:] == 77).all(), s


# ----------------------------------------------------- strides, streams, graphs
@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_strided_rows(env, form):
    """Q as a slice of a joint q/k/v array, O as a slice of a wider one."""
    torch, slim = env
    c = case(torch, 31, "bf16", [33, 100, 64], 4, 2, 96, 16, new=None if form == "decode" else [33, 5, 64])
    want = run(env, c)
    tokens = c["q"].shape[0]
    joint = torch.randn(tokens, 8, 96, device="cuda").bfloat16()
    joint[:, 2:6] = c["q"]
    wide = torch.full((tokens, 7, 96), 77.0, device="cuda", dtype=torch.bfloat16)
    c2 = dict(c, q=joint[:, 2:6])
    got = run(env, c2, out=wide[:, 1:5])
    assert torch.equal(got, want)
    assert (wide[:, :1] == 77).all() and (wide[:, 5:] == 77).all()


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_repeats_bit_for_bit_on_one_workspace_and_other_streams(env, form):
    torch, slim = env
    ws = None
    first = {}
    side = torch.cuda.Stream()
    for turn in range(3):
        for i, (lens, new) in enumerate([([3000, 10], [1, 3]), ([5], [5]), ([100] * 40, [7] * 40)]):
            c = case(torch, 40 + i, "fp16", lens, 4, 2, 128, 64, new=None if form == "decode" else new)
            if ws is None:
                ws = slim.workspace_attention(400, 400, 8, 4, 256)
            y = run(env, c, ws=ws).clone()
            if turn == 0:
                check(c, y)
                first[i] = y
            else:
                assert torch.equal(y, first[i])
            torch.cuda.synchronize()
            y = torch.empty_like(c["q"])
            z = run(env, c, out=y, stream=side)              # workspace made by the call, on that stream
            side.synchronize()
            assert torch.equal(z, first[i])


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_graph_replays_follow_the_device_arrays(env, form):
    """One captured call serves lengths, tables and queries that change between replays."""
    torch, slim = env
    new = None if form == "decode" else [3, 20]
    cs = [case(torch, 50 + i, "fp16", lens, 4, 2, 128, 16, new=new, width=80, pages=200)
          for i, lens in enumerate([[40, 700], [1000, 41], [20, 1280], [3, 20]])]
    st = {n: cs[0][n].clone() for n in ("q", "k", "v", "d_table", "d_lens")}
    st.update(scale=cs[0]["scale"], starts=cs[0]["starts"], d_starts=cs[0]["d_starts"])
    ws = slim.workspace_attention(st["q"].shape[0], 2, 4, 2, 128)
    out = torch.empty_like(st["q"])
    run(env, st, ws=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if new is None:
            slim.attention_decode(st["q"], st["k"], st["v"], st["d_table"], st["d_lens"], scale=st["scale"], ws=ws, out=out)
        else:
            slim.attention_prefill(st["q"], st["k"], st["v"], st["d_table"], st["d_lens"], st["d_starts"],
                                   scale=st["scale"], ws=ws, out=out)
    for turn in range(2):
        for c in cs:
            for n in ("q", "k", "v", "d_table", "d_lens"):
                st[n].copy_(c[n])
            out.fill_(77.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            check(c, out, what=f"replay {turn}")
            assert torch.equal(out, run(env, c, ws=ws)), "replay differs from the eager call"


def test_offsets_past_32_bits(env):
    """Pages whose element and byte offsets pass 2^31 and 2^32."""
    torch, slim = env
    kv_heads, page, dim = 8, 64, 128
    pages = (5 << 30) // (kv_heads * page * dim) + 7              # 5 * 2^30 elements, 10 GiB
    kpool = torch.empty((pages, kv_heads, page, dim), dtype=torch.float16, device="cuda")
    vpool = torch.empty_like(kpool)
    c = case(torch, 61, "fp16", [200, 130], 16, kv_heads, dim, page, new=None, pages=8)
    far = [pages - 1 - 3 * i for i in range(8)] if pages > 30 else None
    near = list(range(8))
    table = np.where(c["table"] >= 0, np.asarray(far)[np.maximum(c["table"], 0)], -1).astype(np.int32)
    d_table = torch.from_numpy(table).cuda()
    for p, f in zip(near, far):
        kpool[f].copy_(c["k"][p])
        vpool[f].copy_(c["v"][p])
    c2 = dict(c, k=kpool, v=vpool, d_table=d_table)
    assert torch.equal(run(env, c2), run(env, c)), "decode"
    q = torch.randn(40, 16, dim, device="cuda").half()
    starts = torch.tensor([0, 33, 40], dtype=torch.int32, device="cuda")
    a = slim.attention_prefill(q, c["k"], c["v"], c["d_table"], c["d_lens"], starts)
    b = slim.attention_prefill(q, kpool, vpool, d_table, c["d_lens"], starts)
    assert torch.equal(a, b), "prefill"
    # Append to and copy between far pages.
    k_new = torch.randn(2, kv_heads, dim, device="cuda").half()
    slim.kv_append(k_new, -k_new, kpool, vpool, d_table, c["d_lens"])
    for s, n in enumerate((200, 130)):
        p, r = int(table[s, (n - 1) // page]), (n - 1) % page
        assert torch.equal(kpool[p, :, r], k_new[s]) and torch.equal(vpool[p, :, r], -k_new[s])
    src = torch.tensor([far[0], 5], dtype=torch.int32, device="cuda")
    dst = torch.tensor([11, far[0] - 1], dtype=torch.int32, device="cuda")
    kpool[5].fill_(3.0)
    vpool[5].fill_(4.0)
    slim.kv_copy_pages(kpool, vpool, src, dst)
    assert torch.equal(kpool[11], kpool[far[0]]) and torch.equal(vpool[11], vpool[far[0]])
    assert (kpool[far[0] - 1] == 3).all() and (vpool[far[0] - 1] == 4).all()


# ------------------------------------------------------------ larger grids
@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("fp16", 128), ("bf16", 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5), (500, 0)])
def test_prefill_more_row_blocks_than_a_round_of_workgroups(env, dtype, dim, window, sinks):
    """Many short sequences with one behind a prefix of more than 64 tiles, unsplit."""
    new = [3] + [int(n) for n in np.random.default_rng(71).integers(0, 9, 70)]
    pre = [9000] + [int(n) for n in np.random.default_rng(72).integers(0, 150, 70)]
    c = case(env[0], 71, dtype, [n + p for n, p in zip(new, pre)], 8, 4, dim, 32, new=new)
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_long_unsplit_walk_of_both_wave_groups(env, dim):
    """As few row blocks as one round holds, unsplit: each group of waves walks more than 64 tiles."""
    new = [2] + [1] * 45
    pre = [9500] + [int(n) for n in np.random.default_rng(73).integers(0, 200, 45)]
    c = case(env[0], 73, "fp16", [n + p for n, p in zip(new, pre)], 4, 4, dim, 16, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("q_heads,kv_heads,new,pre", [(12, 4, 700, 0), (4, 4, 600, 333), (64, 8, 130, 40), (7, 7, 129, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 3)])
def test_prefill_row_blocks_cross_tokens_and_heads(env, q_heads, kv_heads, new, pre, window, sinks):
    c = case(env[0], 74, "bf16", [new + pre, 5], q_heads, kv_heads, 64, 64, new=[new, 2])
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


def test_seen_infinities_give_what_the_formula_gives(env):
    """An infinite value reaches the rows that see it, in its element only; an infinite score gives NaN."""
    torch, slim = env
    for new in (None, [90]):
        c = case(torch, 75, "bf16", [90], 2, 1, 64, 16, new=new)
        k, v = host(c["k"]), host(c["v"])
        want, _, mass = reference(c, k=k, v=v)
        page = int(c["table"][0, 4])
        c["v"][page, 0, 6, 3] = float("inf")                      # key 70
        got = host(run(env, c))
        assert np.isposinf(got[-1, :, 3]).all()
        rows = np.arange(got.shape[0]) if new else np.asarray([89])
        for t, p in enumerate(rows):
            keep = np.arange(64) != 3 if p >= 70 else np.ones(64, dtype=bool)
            over = np.abs(got[t][:, keep] - want[t][:, keep]) - bound(c, want[t], mass[t])[:, keep]
            assert over.max() <= 0, (p, over.max())
        c["v"][page, 0, 6, 3] = 0.0
        c["q"][-1, 0, 0] = float("inf")
        assert np.isnan(host(run(env, c))[-1, 0]).all()

"""slim_attention_prefill_q4 on both of its ways: a few new rows a sequence (16 at
a time, as single tokens) and many (128 at a time), at the border between them, and
where rows of one block see different keys."""
import numpy as np
import pytest

from attention_helpers import bound, check, host, reference
from q4_helpers import junk_rows, q4_case, scale_byte
from test_attention_q4_gpu import DTYPES, HEADS, WINDOWS, env, run  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ few rows
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [*HEADS, (4, 4), (9, 3)])
def test_few_rows_head_layouts(env, dtype, dim, q_heads, kv_heads):
    lens = [1, 40, 130, 0, 17, 300, 33]
    new = [1, 0, 2, 0, 1, 0, 3] if q_heads // kv_heads > 8 else [1, 3, 0, 0, 17, 5, 4]
    c = q4_case(env[0], 61, dtype, lens, q_heads, kv_heads, dim, 16, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 128), ("bf16", 96), ("fp16", 256)])
def test_few_rows_window_and_sinks(env, dtype, dim, window, sinks):
    c = q4_case(env[0], 62, dtype, [300, 1, 500, 700, 12], 4, 2, dim, 16, new=[40, 1, 20, 9, 12])
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("bf16", 128), ("fp16", 256)])
@pytest.mark.parametrize("seqs,q_heads,kv_heads,longest,most", [(1, 8, 1, 6000, 6), (1, 32, 8, 2500, 9), (4, 8, 8, 1500, 16),
                                                                (20, 16, 16, 400, 5), (70, 8, 8, 200, 3)])
def test_few_rows_every_plan(env, dtype, dim, seqs, q_heads, kv_heads, longest, most):
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, longest + 1, seqs)
    lens[-1] = longest
    new = np.minimum(rng.integers(0, most + 1, seqs), lens)
    new[-1] = most
    c = q4_case(env[0], 63, dtype, [int(n) for n in lens], q_heads, kv_heads, dim, 64, new=[int(n) for n in new])
    want, want_lse, mass = reference(c)
    limit, seen = bound(c, want, mass), ~np.isneginf(want_lse)
    for max_len in (None, 0, 300, 1500, 9000, 200000):
        y, lse = run(env, c, lse=True, max_len=max_len)
        y, lse = host(y), host(lse)
        assert (np.abs(y - want) <= limit).all(), f"max_len={max_len}"
        # (The bound of attention_helpers.check.)
        assert np.array_equal(~np.isneginf(lse), seen) and (np.abs(lse[seen] - want_lse[seen]) <= 2.0 ** -12 * (
            1 + np.abs(want_lse[seen]).max(initial=0.0))).all(), f"max_len={max_len}: lse"


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 128), ("fp16", 96), ("bf16", 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_few_rows_later_nan_keys_do_not_reach_earlier_rows(env, dtype, dim, window, sinks):
    torch, slim = env
    c = q4_case(torch, 64, dtype, [150, 40], 2, 1, dim, 16, new=[22, 1])
    at = (140, 147, 149)
    clean, _, mass = reference(c, window, sinks)
    for j in at:
        for pool in ("k4", "v4"):
            scale_byte(c[pool], int(c["table"][0, j // 16]), 0, j % 16, 1).fill_(255)
    got = host(run(env, c, window, sinks))
    for i in range(23):
        p = 128 + i if i < 22 else -1
        if any(j <= p for j in at):
            assert np.isnan(got[i]).all()
            continue
        assert ((np.abs(got[i] - clean[i]) - bound(c, clean[i], mass[i])) <= 0).all(), f"row {i}"


@pytest.mark.parametrize("junk", ["any", "nan", "max"])
@pytest.mark.parametrize("dtype,dim", [("fp16", 128), ("bf16", 96), ("bf16", 64), ("fp16", 256)])
def test_few_rows_unseen_places_do_not_reach_a_row(env, dtype, dim, junk):
    torch, slim = env
    c = q4_case(torch, 65, dtype, [70, 9, 333, 200], 4, 2, dim, 16, new=[7, 1, 33, 20])
    scale = {"any": None, "nan": 255, "max": 254}[junk]
    rng = np.random.default_rng(65)
    owned = {}
    for b in range(4):
        for j in range(int(c["lens"][b])):
            owned.setdefault(int(c["table"][b, j // 16]), set()).add(j % 16)
    for p in range(c["k"].shape[0]):
        for pool in ("k4", "v4"):
            junk_rows(torch, c[pool], p, [r for r in range(16) if r not in owned.get(p, ())], rng, scale)
    check(c, run(env, c), what="unowned places")
    window, sinks = 40, 2
    for j in range(sinks, 333 - 33 - window + 1):
        for pool in ("k4", "v4"):
            junk_rows(torch, c[pool], int(c["table"][2, j // 16]), [j % 16], rng, scale)
    check(c, run(env, c, window, sinks), window=window, sinks=sinks, what="outside the window")


@pytest.mark.parametrize("skip,cut", [(0, 5), (7, 0), (13, 16), (1, 0), (0, 1)])
@pytest.mark.parametrize("lens,new", [([300, 200], [20, 17]), ([5000, 4100], [20, 17])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_few_rows_of_a_part_of_the_tokens(env, lens, new, skip, cut, window, sinks):
    """Starts that begin before row 0 or end past the last one."""
    torch, slim = env
    c = q4_case(torch, 66, "bf16", lens, 2, 1, 128, 16, new=new)
    rows = slice(skip, sum(new) - cut)
    q = c["q"][rows]
    out = torch.full_like(q, 77.0)
    slim.attention_prefill_q4(q, c["k4"], c["v4"], c["d_table"], c["d_lens"], c["d_starts"] - skip, window=window, sinks=sinks,
                              scale=c["scale"], out=out)
    torch.cuda.synchronize()
    want, _, mass = (x[rows] for x in reference(c, window, sinks))
    assert ((np.abs(host(out) - want) - bound(c, want, mass)) <= 0).all()


@pytest.mark.parametrize("starts", [[-2 ** 31, -5, 20], [-2 ** 31, 20, 2 ** 31 - 1], [0, 10, 2 ** 31 - 1], [-300, 12, 500]])
def test_few_rows_far_starts(env, starts):
    torch, slim = env
    c = q4_case(torch, 67, "fp16", [300, 250], 2, 1, 64, 16, new=[15, 15])
    out = torch.full_like(c["q"], 77.0)
    slim.attention_prefill_q4(c["q"], c["k4"], c["v4"], c["d_table"], c["d_lens"],
                              torch.tensor(starts, dtype=torch.int32, device="cuda"), scale=c["scale"], out=out)
    torch.cuda.synchronize()
    got = host(out)
    for t in range(30):
        b = next((b for b in range(2) if starts[b] <= t < starts[b + 1]), None)
        if b is None:
            assert (got[t] == 77).all()
            continue
        at = int(c["lens"][b]) - (starts[b + 1] - t) + 1        # keys that the row sees
        if at <= 0:
            assert (got[t] == 0).all()
            continue
        one = dict(c, q=c["q"][t:t + 1], table=c["table"][b:b + 1], lens=np.asarray([at]), starts=None)
        want, _, mass = reference(one)
        assert ((np.abs(got[t] - want[0]) - bound(one, want[0], mass[0])) <= 0).all()


@pytest.mark.parametrize("lens,new", [([5000], [4]), ([9000, 300], [3, 0]), ([40, 70], [2, 7])])
def test_few_rows_among_rows_of_no_sequence(env, lens, new):
    torch, slim = env
    c = q4_case(torch, 73, "fp16", lens, 4, 2, 64, 16, new=new)
    q = torch.cat([c["q"][:1], c["q"], c["q"][:2]])
    out = torch.full_like(q, 77.0)
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    slim.attention_prefill_q4(q, c["k4"], c["v4"], c["d_table"], c["d_lens"], c["d_starts"] + 1, scale=c["scale"], out=out, lse=lse)
    torch.cuda.synchronize()
    n = sum(new)
    check(c, out[1:n + 1], lse[1:n + 1])
    for x in (out, lse):
        assert (x[:1] == 77).all() and (x[n + 1:] == 77).all()


def test_few_rows_scale_and_peaked_scores(env):
    c = q4_case(env[0], 68, "fp16", [700, 64, 9], 4, 2, 128, 16, new=[9, 2, 9], q_std=3.0)
    check(c, run(env, c))
    c["scale"] = -c["scale"]
    check(c, run(env, c), what="negative scale")
    c["scale"] = 0.0
    check(c, run(env, c), what="scale 0: the mean of the values")


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 128), ("bf16", 96), ("fp16", 256)])
@pytest.mark.parametrize("q_heads,kv_heads,new", [(4, 2, [20, 1, 20, 9, 12]), (40, 1, [1, 0, 2, 0, 0]), (8, 8, [30, 1, 32, 40, 12])])
def test_few_rows_windows_of_other_heads(env, dtype, dim, q_heads, kv_heads, new):
    c = q4_case(env[0], 70, dtype, [300, 1, 500, 700, 12], q_heads, kv_heads, dim, 16, new=new)
    for window, sinks in [(0, 0), *WINDOWS]:
        y, lse = run(env, c, window, sinks, lse=True)
        check(c, y, lse, window, sinks)


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("bf16", 128), ("fp16", 256)])
@pytest.mark.parametrize("q_heads,kv_heads,new", [(8, 1, 4), (32, 8, 7), (3, 3, 29)])
def test_few_rows_of_one_sequence_split(env, dtype, dim, q_heads, kv_heads, new):
    c = q4_case(env[0], 72, dtype, [5000], q_heads, kv_heads, dim, 64, new=[new])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    y, lse = run(env, c, 3000, 9, lse=True, max_len=200000)
    check(c, y, lse, 3000, 9)


# --------------------------------------------------------- the border, many rows
@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 128)])
@pytest.mark.parametrize("new", [[64, 0], [65, 0], [32, 32], [31, 34], [96, 0], [97, 0], [48, 48], [47, 50], [1, 200], [90, 1, 1, 1, 200, 1, 1, 1]])
def test_around_the_border(env, dtype, dim, new):
    c = q4_case(env[0], 69, dtype, [n + 100 for n in new], 3, 3, dim, 32, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    y, lse = run(env, c, 50, 3, lse=True)
    check(c, y, lse, 50, 3)


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("fp16", 128), ("bf16", 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 5)])
def test_many_rows_more_blocks_than_a_round_of_workgroups(env, dtype, dim, window, sinks):
    """Sequences of some 50 rows with one behind a prefix of more than 64 tiles, unsplit: pages are looked up again on the way."""
    new = [30] + [int(n) for n in np.random.default_rng(71).integers(40, 62, 70)]
    pre = [9000] + [int(n) for n in np.random.default_rng(72).integers(0, 50, 70)]
    c = q4_case(env[0], 71, dtype, [n + p for n, p in zip(new, pre)], 4, 4, dim, 32, new=new)
    y, lse = run(env, c, window, sinks, lse=True)
    check(c, y, lse, window, sinks)


@pytest.mark.parametrize("dtype,dim", [("fp16", 64), ("bf16", 96), ("bf16", 128), ("fp16", 256)])
def test_many_rows_long_unsplit_walk_of_both_wave_groups(env, dtype, dim):
    new = [60] + [50] * 41
    pre = [9500] + [int(n) for n in np.random.default_rng(73).integers(0, 200, 41)]
    c = q4_case(env[0], 73, dtype, [n + p for n, p in zip(new, pre)], 4, 4, dim, 16, new=new)
    y, lse = run(env, c, lse=True)
    check(c, y, lse)


@pytest.mark.parametrize("q_heads,kv_heads", [(2, 2), (8, 1)])
def test_many_rows_on_a_long_prefix(env, q_heads, kv_heads):
    c = q4_case(env[0], 74, "bf16", [6063, 4000 + 17, 9050], q_heads, kv_heads, 128, 64, new=[63, 90, 50])
    y, lse = run(env, c, lse=True)
    check(c, y, lse)
    check(c, run(env, c, window=1000, sinks=4), window=1000, sinks=4)
    for max_len in (0, 1, 1 << 30):
        check(c, run(env, c, max_len=max_len), what=f"max_len={max_len}")

"""Inputs and the error bound of the attention tests."""
import numpy as np

from oracle import attention_ref as ref

# Unit roundoff of the half types (10 and 7 stored mantissa bits).
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def case(torch, seed, dtype, lens, q_heads, kv_heads, dim, page, new=None, spare=3, q_std=1.0, width=None, pages=None):
    """Random pools, a table of scattered pages and queries on the GPU, the
    values of all of them on the host in fp64.  `new`: new tokens per sequence
    (None: single-token form, no starts)."""
    rng = np.random.default_rng(seed)
    td = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    used = [-(-max(n, 0) // page) for n in lens]
    width = max(max(used, default=0), 1) if width is None else width
    pages = sum(used) + spare if pages is None else pages
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :min(n, width)] = order[at:at + min(n, width)]
        at += n
    starts = None if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tokens = len(lens) if new is None else int(starts[-1])

    def half(*shape, std=1.0):
        return (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)) * std).to(td).cuda()

    c = dict(q=half(tokens, q_heads, dim, std=q_std), k=half(pages, kv_heads, page, dim),
             v=half(pages, kv_heads, page, dim), table=table, lens=np.asarray(lens, dtype=np.int32), starts=starts,
             dtype=dtype, scale=dim ** -0.5)
    c["d_table"] = torch.from_numpy(table).cuda()
    c["d_lens"] = torch.from_numpy(c["lens"]).cuda()
    c["d_starts"] = None if starts is None else torch.from_numpy(starts).cuda()
    return c


def host(t):
    return t.double().cpu().numpy()


def reference(c, window=0, sinks=0, k=None, v=None):
    return ref.attention(host(c["q"]), host(c["k"]) if k is None else k, host(c["v"]) if v is None else v, c["table"],
                         c["lens"], c["starts"], c["scale"], window, sinks)


def bound(c, out, mass):
    """How far an output may be from the fp64 one.  With u the type's unit
    roundoff, |o| u for the output's own rounding; each weight rounded once to
    the type before the product with v: mass * u, and 2^-24 |v| n for weights
    below the type's normal range (n keys, sum at least 1); scores, exponentials
    and sums in fp32: a score of dim products is off by at most dim 2^-24 times
    its sum of magnitudes, which N(0, 1) operands keep under 8 sqrt(dim) * scale
    * std = 8 std, so weights by twice that plus the sum's own n 2^-24, all under 2^-12
    * mass at the lengths tested.  A tenth is added for second-order terms."""
    u = UNIT[c["dtype"]]
    return 1.1 * (np.abs(out) * u + mass * (u + 2.0 ** -12)) + 2.0 ** -20


def check(c, got, lse=None, window=0, sinks=0, what="", **kw):
    out, ref_lse, mass = reference(c, window, sinks, **kw)
    got = host(got)
    assert got.shape == out.shape
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - out) - bound(c, out, mass)
    assert over.max(initial=-1.0) <= 0, f"{what}: {over.max():.3e} beyond the bound, at {np.unravel_index(over.argmax(), over.shape)}"
    if lse is not None:
        lse = host(lse)
        assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse)), f"{what}: lse of empty rows"
        fine = ~np.isneginf(ref_lse)
        assert np.abs(lse[fine] - ref_lse[fine]).max(initial=0.0) <= 2.0 ** -12 * (1 + np.abs(ref_lse[fine]).max(initial=0.0)), f"{what}: lse"

"""Cases of the rotary positions and the 4-bit key-value cache, and their plain forms.

What lies between a decoder block's q/k/v projections and its paged cache, and
the attention over that cache where it holds 4 bits a value: the rotation of
rows by their positions ("rope"), the writing of new keys and values to their
pages with the keys (and the step's queries) rotated on the way
("append_rope"), the same into pages of 4 bits ("append_q4"; the new tokens are
read back, as the values that the codes stand for), and attention over such
pages for single tokens ("decode_q4") and for prompts and chunks of prompts
("prefill_q4").

The 4-bit format.  A key or value row of one head is cut into groups of 32; a
group is 32 codes (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2,
3, 4 or 6) times 2^e, e the smallest whole number for which no element
exceeds 7 * 2^e, held within the type's range; a value goes to the nearest code,
ties to the even one, 6 at most.  A page is uint8 [kv_heads, page, dim * 17/32], in it
first all codes [kv_heads][page][dim / 2] (element 2 i in the low four bits
of byte i), then all e + 127 as bytes [kv_heads][page / 16][dim / 32][16].

A case is a dict; its lengths follow from its numbers alone (``_lens``), the
values of its tensors from the seed.  ``own`` selects the framework's kernels
instead of the plain torch form.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
# Least and largest e of a group: half of 2^e is the least number of the type that counts (fp16's subnormals do), and
# 6 * 2^e is finite.
EXPONENTS = {"fp16": (-23, 13), "bf16": (-125, 125)}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The queries of one new token: launch latency counts.
        _rope("rope 1 token", "bf16", 1, 32, 128, 128, False, "none", 4000),
        # The queries of a long prompt, half of each head rotated, interleaved pairs, positions far past the trained ones.
        _rope("rope 4099 tokens far", "fp16", 4099, 32, 128, 64, True, "yarn", 120000),
        # The cache's share of one decode step of a batch, keys and queries rotated on the way.
        _append("append_rope", "append_rope 64 x 1", "fp16", 64, 1, 1, 1, 4000, 32, 32, 128, 64, 128, False, "none"),
        # The same for eight prompts behind cached prefixes, grouped heads, positions scaled.
        _append("append_rope", "append_rope 8 x 300..1900", "bf16", 8, 300, 1900, 0, 700, 32, 8, 128, 16, 128, False,
                "linear"),
        # The decode step's append into pages of 4 bits.
        _append("append_q4", "append_q4 64 x 1", "bf16", 64, 1, 1, 1, 4000, 32, 8, 128, 64, 128, False, "ntk"),
        # Eight prompts into pages of 4 bits, one key head per query head.
        _append("append_q4", "append_q4 8 x 300..1900", "fp16", 8, 300, 1900, 0, 700, 32, 32, 128, 64, 128, True, "none"),
        # The first step of a chat turn: one sequence, a handful of cached tokens.
        _decode("decode_q4 1 x 33", "fp16", 1, 33, 33, 32, 32, 128, 16),
        # A serving batch of mixed ages, one key head per query head (4096 = 32 heads of 128).
        _decode("decode_q4 64 x 1..4096", "fp16", 64, 1, 4096, 32, 32, 128, 64),
        # One long document: few rows, a long axis; four query heads share a key head.
        _decode("decode_q4 1 x 131071 grouped", "bf16", 1, 131071, 131071, 32, 8, 128, 128),
        # A batch of long conversations with a sliding window and four first tokens kept.
        _decode("decode_q4 32 x 9..32768 window", "bf16", 32, 9, 32768, 32, 8, 64, 64, window=4096, sinks=4),
        # A chunk of a prompt behind a long cached prefix: few query rows, a long axis.
        _prefill("prefill_q4 61 on 24576", "bf16", 1, 61, 61, 24576, 24576, 32, 8, 128, 64),
        # Prompts of odd sizes, some behind cached prefixes.
        _prefill("prefill_q4 4 x 700..4096", "fp16", 4, 700, 4096, 0, 1500, 32, 8, 128, 64),
    ]


def _rope(name, dtype, tokens, heads, dim, rot, interleaved, scaling, most):
    return {"name": name, "op": "rope", "dtype": dtype, "tokens": tokens, "heads": heads, "dim": dim, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "most": most}


def _append(op, name, dtype, seqs, lo, hi, pre_lo, pre_hi, q_heads, kv_heads, dim, page, rot, interleaved, scaling):
    return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "new_lo": lo, "new_hi": hi, "pre_lo": pre_lo,
            "pre_hi": pre_hi, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "rot": rot,
            "interleaved": interleaved, "scaling": scaling}


def _decode(name, dtype, seqs, lo, hi, q_heads, kv_heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "decode_q4", "dtype": dtype, "seqs": seqs, "len_lo": lo, "len_hi": hi,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "sinks": sinks}


def _prefill(name, dtype, seqs, lo, hi, pre_lo, pre_hi, q_heads, kv_heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "prefill_q4", "dtype": dtype, "seqs": seqs, "new_lo": lo, "new_hi": hi,
            "pre_lo": pre_lo, "pre_hi": pre_hi, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "window": window, "sinks": sinks}


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    dtype = rng.choice(("fp16", "bf16"))
    dim = rng.choice((64, 96, 128, 128, 128, 256))
    page = rng.choice((16, 32, 64, 128))
    q_heads, kv_heads = rng.choice(((32, 32), (32, 8), (32, 4), (64, 8), (28, 4), (12, 12), (20, 1)))
    rot = rng.choice((dim, dim, dim // 2, dim // 4))
    interleaved = rng.random() < 0.5
    scaling = rng.choice(("none", "linear", "ntk", "yarn"))
    op = rng.choice(("rope", "append_rope", "append_q4", "decode_q4", "decode_q4", "prefill_q4", "prefill_q4"))
    if op == "rope":
        most = (1 << 24) // (q_heads * dim)
        case = _rope("", dtype, log_int(1, min(8192, most)), q_heads, dim, rot, interleaved, scaling, log_int(1, 1 << 20))
    elif op.startswith("append"):
        seqs = log_int(1, 128)
        hi = log_int(1, max(1, min(8192, (1 << 25) // (kv_heads * dim)) // seqs))
        pre = log_int(1, 4096)
        case = _append(op, "", dtype, seqs, rng.randint(1, hi), hi, rng.randint(0, pre), pre, q_heads, kv_heads, dim, page,
                       rot, interleaved, scaling)
    else:
        window = rng.choice((0, 0, log_int(16, 8192)))
        sinks = rng.choice((0, 1, 4, 64)) if window else 0
        if op == "decode_q4":
            seqs = log_int(1, 128)
            hi = log_int(1, max(1, min(131072, (1 << 31) // (seqs * kv_heads * dim * 4))))
            case = _decode("", dtype, seqs, rng.randint(1, hi), hi, q_heads, kv_heads, dim, page, window, sinks)
        else:
            seqs = log_int(1, 16)
            # Query rows x keys, over all heads, up to a 4096-token prompt of 32 heads of 128.
            most = (1 << 24) * 32 * 128 // (q_heads * dim * seqs)
            pre = rng.choice((0, 0, log_int(1, 24576)))
            hi = log_int(1, min(6000, int(math.sqrt(most + pre * pre / 4.0) - pre / 2.0)))
            case = _prefill("", dtype, seqs, rng.randint(1, hi), hi, rng.randint(0, pre), pre, q_heads, kv_heads, dim,
                            page, window, sinks)
    del case["name"]
    return case


def _lens(lo, hi, count):
    """``count`` lengths from lo to hi, both ends among them where count > 1."""
    if count == 1:
        return [hi]
    return [lo, hi] + [lo + int((hi - lo) * math.modf(0.6180339887498949 * (i + 1))[0]) for i in range(count - 2)]


def _rows(case):
    """(new tokens, cached tokens with the new ones) of every sequence."""
    if case["op"] == "decode_q4":
        lens = _lens(case["len_lo"], case["len_hi"], case["seqs"])
        return [1] * len(lens), lens
    new = _lens(case["new_lo"], case["new_hi"], case["seqs"])
    pre = _lens(case["pre_lo"], case["pre_hi"], case["seqs"])[::-1]
    return new, [n + p for n, p in zip(new, pre)]


def _rope_args(case):
    """What a program says of its rotation: a model trained on 4096 positions, stretched by 4 where it is scaled."""
    args = {"rot_dim": case["rot"], "base": 10000.0, "interleaved": case["interleaved"]}
    if case["scaling"] != "none":
        args.update(scaling=case["scaling"], factor=4.0)
    if case["scaling"] == "yarn":
        args["original_len"] = 4096
    return args


def _frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, **_):
    """(radians a position of every pair, factor of the rotated elements).  "linear" divides positions by `factor`;
    "ntk" stretches the base so that the slowest pair turns `factor` times slower; "yarn" slows the pairs that turn less
    than once in original_len, leaves those that turn 32 times and more, and blends between; its rotated elements are
    multiplied by 0.1 ln(factor) + 1."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def pair_of(turns):          # the pair (a real number) that turns so often in original_len positions
        return rot * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

    low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rot - 1)
    slow = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
    return f * (1.0 - slow) + f / factor * slow, 0.1 * math.log(factor) + 1.0


def _rope_of(case):
    """What a program makes once for its model."""
    import sparse_int4_gemm_amd as slim

    return slim.Rope(**_rope_args(case), device="cuda")


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    state = {"case": case}
    if "rot" in case:
        args = _rope_args(case)
        freqs, state["magnitude"] = _frequencies(args.pop("rot_dim"), **args)
        state["freqs"] = freqs.to(dev)
        state["rope"] = _rope_of(case) if own else None
    if case["op"] == "rope":
        n, most = case["tokens"], case["most"]
        first = int(torch.randint(0, max(1, most - n + 1), (1,), generator=gen, device=dev))
        state["x"] = normal(n, case["heads"], case["dim"])
        state["positions"] = torch.arange(first, first + n, device=dev, dtype=torch.int32)
        state["out"] = torch.empty_like(state["x"])
        return state

    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    new, lens = _rows(case)
    width = -(-max(lens) // page)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 3
    # Every sequence's pages lie anywhere in the pool, as after many requests; entries past its end are not used.
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    tokens = starts[-1]
    state.update(table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
                 starts=torch.tensor(starts, dtype=torch.int32, device=dev), tokens=tokens, max_len=max(lens),
                 max_new=max(new))
    if case["op"] == "append_rope":
        state["k"], state["v"] = normal(pages, heads, page, dim), normal(pages, heads, page, dim)
    elif case["op"] == "append_q4":
        state["k"], state["v"] = (torch.zeros((pages, heads, page, dim * 17 // 32), dtype=torch.uint8, device=dev)
                                  for _ in range(2))
    else:
        state["k"], state["v"] = (torch.empty((pages, heads, page, dim * 17 // 32), dtype=torch.uint8, device=dev)
                                  for _ in range(2))
        step = max(1, (1 << 27) // (heads * page * dim))
        for pool in (state["k"], state["v"]):
            for a in range(0, pages, step):
                codes, scales = _parts(pool[a:a + step], case)
                code, e = _quantise(normal(codes.shape[0], heads, page, dim).float(), case["dtype"])
                codes.copy_(code[..., 0::2] | code[..., 1::2] << 4)
                scales.copy_(e.view(-1, heads, page // 16, 16, dim // 32).transpose(3, 4))
    state["q"] = normal(tokens, case["q_heads"], dim)
    # What a serving program allocates once for its batch.
    state["out"] = torch.empty_like(state["q"])
    if "rot" in case:
        state["new_k"], state["new_v"] = normal(tokens, heads, dim), normal(tokens, heads, dim)
    else:
        state["scale"] = 1.0 / math.sqrt(dim)
        state["ws"] = {}
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import sparse_int4_gemm_amd as slim

    case = s["case"]
    op = case["op"]
    if "rope" in s and s["rope"] is None:
        s["rope"] = _rope_of(case)
    if op == "rope":
        return slim.rope(s["x"], s["positions"], s["rope"], out=s["out"])
    if op == "append_rope":
        slim.kv_append_rope(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["lens"], s["rope"],
                            starts=s["starts"], q=s["q"], q_out=s["out"])
        return [s["out"], s["k"], s["v"]]
    if op == "append_q4":
        slim.kv_append_q4(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["lens"], starts=s["starts"],
                          rope=s["rope"], q=s["q"], q_out=s["out"])
        return [s["out"], *slim.kv_read_q4(s["k"], s["v"], s["table"], s["lens"], starts=s["starts"],
                                           tokens=s["tokens"], dtype=s["q"].dtype)]
    if not s["ws"]:
        s["ws"]["ws"] = slim.workspace_attention(s["tokens"], case["seqs"], case["q_heads"], case["kv_heads"],
                                                 case["dim"])
    kw = dict(max_len=s["max_len"], window=case["window"], sinks=case["sinks"], scale=s["scale"], ws=s["ws"]["ws"],
              out=s["out"])
    if op == "decode_q4":
        return slim.attention_decode_q4(s["q"], s["k"], s["v"], s["table"], s["lens"], **kw)
    return slim.attention_prefill_q4(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], **kw)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        cos, sin = _angles(s, s["positions"])
        return _turn(s["x"].float(), cos.float(), sin.float(), case["interleaved"]).to(s["x"].dtype)
    # Sequence and position of every token, then the place of that position in the pool.
    starts, lens, page = s["starts"].long(), s["lens"].long(), case["page"]
    token = torch.arange(s["tokens"], device=starts.device)
    seq = (token[:, None] >= starts[None, 1:]).sum(1)
    row = token - starts[seq]
    pos = lens[seq] - (starts[seq + 1] - starts[seq]) + row
    if op in ("decode_q4", "prefill_q4"):
        return _attention_plain(s, seq, row, pos)
    at = s["table"].long()[seq, pos // page]
    cos, sin = _angles(s, pos)
    q = _turn(s["q"].float(), cos.float(), sin.float(), case["interleaved"]).to(s["q"].dtype)
    if op == "append_rope":
        k = _turn(s["new_k"].float(), cos.float(), sin.float(), case["interleaved"])
        s["k"][at, :, pos % page] = k.to(s["k"].dtype)
        s["v"][at, :, pos % page] = s["new_v"]
        return [q, s["k"], s["v"]]
    # Values next to a border between two codes: rotated in 64 bits, held in 32.
    k = _turn(s["new_k"].double(), cos, sin, case["interleaved"]).float()
    out = [q]
    for pool, x in ((s["k"], k), (s["v"], s["new_v"].float())):
        code, e = _quantise(x, case["dtype"])
        codes, scales = _parts(pool, case)
        codes[at, :, pos % page] = code[..., 0::2] | code[..., 1::2] << 4
        scales[at, :, pos % page // 16, :, pos % 16] = e
        out.append(_values(code, e).to(s["q"].dtype))
    return out


def _angles(s, positions):
    """Cosines and sines [tokens, 1, pairs] in 64 bits: 32 lose the angles of far positions."""
    angle = positions.double()[:, None, None] * s["freqs"]
    return angle.cos() * s["magnitude"], angle.sin() * s["magnitude"]


def _turn(x, cos, sin, interleaved):
    n = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _parts(pool, case):
    """The codes [pages, heads, page, dim / 2] and exponents [pages, heads, page / 16, dim / 32, 16] of a 4-bit pool (views)."""
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    flat, n = pool.view(pool.shape[0], -1), heads * page * dim // 2
    return (flat[:, :n].view(-1, heads, page, dim // 2), flat[:, n:].view(-1, heads, page // 16, dim // 32, 16))


def _power(e):
    """2^e in 32 bits, e from -126 to 127."""
    return (e.int() + 127 << 23).view(torch.float32)


def _quantise(x, dtype):
    """Codes (uint8, x's shape) and e + 127 (uint8, one for every 32 of the last axis) of x in 32 bits."""
    groups = x.reshape(*x.shape[:-1], -1, 32)
    mantissa, e = torch.frexp(groups.abs().amax(-1))
    e = torch.where(mantissa > 0.875, e - 2, e - 3).clamp_(*EXPONENTS[dtype])
    a = groups * _power(-e[..., None])
    code = (a < 0).to(torch.uint8) << 3
    a = a.abs()
    for i in range(7):
        edge = 0.5 * (LEVELS[i] + LEVELS[i + 1])
        code += a >= edge if i % 2 else a > edge
    return code.view(x.shape), (e + 127).to(torch.uint8)


def _values(code, e):
    """What codes [..., dim] with e + 127 [..., dim / 32] stand for, in 32 bits."""
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), device=code.device)
    x = level[code.int()].view(*code.shape[:-1], -1, 32)
    return (x * _power(e[..., None].int() - 127)).view(code.shape)


def _unpack(pool, case):
    """A 4-bit pool's values [pages, heads, page, dim] in 32 bits."""
    codes, scales = _parts(pool, case)
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return _values(code, scales.transpose(3, 4).reshape(*code.shape[:-1], -1))


def _attention_plain(s, seq, row, pos):
    case = s["case"]
    seqs, new, heads, dim = case["seqs"], s["max_new"], case["kv_heads"], case["dim"]
    share = case["q_heads"] // heads
    # Queries padded to the longest row count: [seqs, heads, new * share, dim]; their positions [seqs, new].
    q = torch.zeros((seqs, new, heads, share, dim), device=s["q"].device)
    q[seq, row] = s["q"].float().view(-1, heads, share, dim)
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs, heads, new * share, dim)
    p = torch.full((seqs, new), -1, device=q.device)
    p[seq, row] = pos
    # Keys and values in the order of the sequences: [seqs, heads, keys, dim].
    table = s["table"].long()
    k, v = (_unpack(pool[table.flatten()], case).view(seqs, -1, heads, case["page"], dim).transpose(1, 2)
            .reshape(seqs, heads, -1, dim) for pool in (s["k"], s["v"]))
    j = torch.arange(k.shape[2], device=q.device)
    seen = j <= p[:, :, None]
    if case["window"]:
        seen &= (j > p[:, :, None] - case["window"]) | (j < case["sinks"])
    seen = seen[:, None, :, None, :]
    scores = torch.matmul(q, k.transpose(2, 3)).view(seqs, heads, new, share, -1).mul_(s["scale"])
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights.view(seqs, heads, new * share, -1), v).view(seqs, heads, new, share, dim)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    out = out.permute(0, 2, 1, 3, 4)[seq, row]
    return out.reshape(-1, heads * share, dim).to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without
def _span(lo, hi, window, sinks):
    """(key-query pairs, different keys) that positions lo .. hi - 1 see."""
    def below(n):      # pairs of positions 0 .. n - 1
        if not window or n <= window:
            return n * (n + 1) // 2
        far = n - window                  # positions window .. n - 1 see `window` recent keys and the sinks before them
        short = min(far, sinks)
        return window * (window + 1) // 2 + far * window + short * (short + 1) // 2 + (far - short) * sinks

    first = max(0, lo - window + 1) if window else 0
    return below(hi) - below(lo), hi - first + min(first, sinks if window else 0)


def work(case):
    size = 2
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    row, held = case["kv_heads"] * case["dim"] * size, case["kv_heads"] * case["dim"] * 17 // 32
    new, lens = _rows(case)
    tokens = sum(new)
    q_row = case["q_heads"] * case["dim"]
    small = 4 * (2 * len(lens) + 1) + 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] in ("append_rope", "append_q4"):
        # New keys and values read, written as they are held, and queries in and out; with 4 bits also what is read back.
        a_row = 2 * row + 2 * row if case["op"] == "append_rope" else 2 * row + 2 * held + 2 * held + 2 * row
        flops = 3 * tokens * (case["q_heads"] + case["kv_heads"]) * case["rot"]
        return {"bytes": tokens * (a_row + 2 * q_row * size) + small + 4 * case["rot"], "flops": flops}
    pairs = keys = 0
    for n, length in zip(new, lens):
        a, b = _span(length - n, length, case["window"], case["sinks"])
        pairs, keys = pairs + a, keys + b
    return {"bytes": 2 * keys * held + 2 * tokens * q_row * size + small, "flops": 4 * pairs * q_row}


# ------------------------------------------------------------------ the definition in 64 bits
def _rotated(x, positions, s):
    """x [tokens, heads, dim] turned as complex numbers."""
    case, n = s["case"], s["case"]["rot"] // 2
    x = x.double()
    pairs = x[..., :2 * n].unflatten(-1, (n, 2)) if case["interleaved"] else x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
    by = torch.polar(torch.full((len(positions), n), float(s["magnitude"]), dtype=torch.float64, device=x.device),
                     torch.outer(positions.double(), s["freqs"]))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by[:, None])
    z = z if case["interleaved"] else z.transpose(-1, -2)
    return torch.cat([z.flatten(-2), x[..., 2 * n:]], -1)


def _held(x, dtype):
    """x in groups of 32, as 4 bits and a power of two hold it."""
    lo, hi = EXPONENTS[dtype]
    groups = x.unflatten(-1, (-1, 32))
    e = torch.ceil(torch.log2(groups.abs().amax(-1, keepdim=True) / 7.0)).clamp(lo, hi)
    a = groups / torch.exp2(e)
    size = a.abs()
    step = torch.where(size < 2.0, 0.5, torch.where(size < 4.0, 1.0, 2.0)).to(a.dtype)
    return (torch.sign(a) * torch.clamp(torch.round(size / step) * step, max=6.0) * torch.exp2(e)).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rotated(s["x"], s["positions"], s)
    new, lens = _rows(case)
    page = case["page"]
    if case["op"] in ("append_rope", "append_q4"):
        positions = torch.cat([torch.arange(m - n, m, device="cuda") for n, m in zip(new, lens)])
        q, k = _rotated(s["q"], positions, s), _rotated(s["new_k"], positions, s)
        if case["op"] == "append_q4":
            # A rotated key is held in 32 bits before it is coded.
            return [q, _held(k.float().double(), case["dtype"]), _held(s["new_v"].double(), case["dtype"])]
        kp, vp, table, at = s["k"].double(), s["v"].double(), s["table"].tolist(), 0
        for b, (n, length) in enumerate(zip(new, lens)):
            i = 0
            while i < n:                                 # as much as the page of this position takes
                pos = length - n + i
                take = min(n - i, page - pos % page)
                for pool, rows in ((kp, k), (vp, s["new_v"].double())):
                    pool[table[b][pos // page], :, pos % page:pos % page + take] = rows[at + i:at + i + take].transpose(0, 1)
                i += take
            at += n
        return [q, kp, vp]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    share, heads, dim, at = case["q_heads"] // case["kv_heads"], case["kv_heads"], case["dim"], 0
    level = torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device="cuda")

    def head_of(pool, ids, h):
        """Keys or values [tokens, dim] of head h in pages ids."""
        flat = pool[ids].view(len(ids), -1)
        codes = flat[:, h * page * dim // 2:(h + 1) * page * dim // 2].reshape(-1, dim // 2)
        first = heads * page * dim // 2 + h * page * dim // 32
        e = flat[:, first:first + page * dim // 32].reshape(-1, dim // 32, 16).transpose(1, 2).reshape(-1, dim // 32)
        x = torch.empty((codes.shape[0], dim), dtype=torch.float64, device="cuda")
        x[:, 0::2], x[:, 1::2] = level[(codes % 16).long()], level[(codes // 16).long()]
        return x * torch.exp2(e.double() - 127.0).repeat_interleave(32, 1)

    for b, (n, length) in enumerate(zip(new, lens)):
        ids = s["table"][b, :-(-length // page)].long()
        i = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hide = j > i
        if case["window"]:
            hide = hide | ((i - j >= case["window"]) & (j >= case["sinks"]))
        for h in range(heads):
            k, v = head_of(s["k"], ids, h)[:length], head_of(s["v"], ids, h)[:length]
            for g in range(h * share, (h + 1) * share):
                a = (s["q"][at:at + n, g].double() @ k.t()) * s["scale"]
                a = torch.softmax(a.masked_fill(hide, -math.inf), dim=1)
                out[at:at + n, g] = a @ v
        at += n
    return out

"""Cases of the attention and cache operators, and their plain forms.

Four operators of a decoder block that lie between its q/k/v and output
projections: attention of one new token over a paged key-value cache
("decode"), attention of prompts and chunks of prompts over that cache, causal,
with an optional sliding window and first tokens that stay visible
("prefill"), the writing of new keys and values to their pages ("append") and
the copying of whole pages in every layer's pool ("copy"; forks and compaction
of a cache).

A case is a dict; its lengths follow from its numbers alone (``_lens``), the
values of its tensors from the seed.  ``own`` selects the framework's kernels
instead of the plain torch form.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The first step of a chat turn: one sequence, a handful of cached tokens.  Launch latency counts.
        _decode("decode 1 x 33", "fp16", 1, 33, 33, 32, 32, 128, 16),
        # A serving batch of mixed ages, one key head per query head (4096 = 32 heads of 128).
        _decode("decode 64 x 1..4096", "fp16", 64, 1, 4096, 32, 32, 128, 64),
        # One long document: few rows, a long axis; four query heads share a key head.
        _decode("decode 1 x 131071 grouped", "bf16", 1, 131071, 131071, 32, 8, 128, 128),
        # A batch of long conversations with a sliding window and four first tokens kept.
        _decode("decode 32 x 9..32768 window", "bf16", 32, 9, 32768, 32, 8, 64, 64, window=4096, sinks=4),
        # A chunk of a prompt behind a long cached prefix: few query rows, a long axis.
        _prefill("prefill 61 on 24576", "bf16", 1, 61, 61, 24576, 24576, 32, 8, 128, 64),
        # One prompt of 2048 tokens, the largest token count of the linear layer's sweep.
        _prefill("prefill 2048", "fp16", 1, 2048, 2048, 0, 0, 32, 32, 128, 64),
        # Prompts of odd sizes, some behind cached prefixes, windowed with sinks.
        _prefill("prefill 8 x 100..2000 window", "bf16", 8, 100, 2000, 0, 1500, 32, 8, 64, 16, window=512, sinks=4),
        # A long prompt under a sliding window of half its length.
        _prefill("prefill 8192 window", "bf16", 1, 8192, 8192, 0, 0, 32, 8, 128, 128, window=4096, sinks=4),
        # The cache's share of one decode step of a batch.
        _append("append 64 x 1", "fp16", 64, 1, 1, 1, 4000, 32, 128, 64),
        # The cache's share of a prefill of eight prompts.
        _append("append 8 x 300..1900", "bf16", 8, 300, 1900, 0, 700, 32, 128, 16),
        # A fork of one sequence: its part-filled last page in all 32 layers.
        _copy("copy 1 page", "fp16", 32, 40, 1, 8, 128, 16),
        # A compaction that moves 45 pages of all 32 layers.
        _copy("copy 45 pages", "bf16", 32, 100, 45, 8, 128, 64),
    ]


def _decode(name, dtype, seqs, lo, hi, q_heads, kv_heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "decode", "dtype": dtype, "seqs": seqs, "len_lo": lo, "len_hi": hi, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "window": window, "sinks": sinks}


def _prefill(name, dtype, seqs, lo, hi, pre_lo, pre_hi, q_heads, kv_heads, dim, page, window=0, sinks=0):
    return {"name": name, "op": "prefill", "dtype": dtype, "seqs": seqs, "new_lo": lo, "new_hi": hi, "pre_lo": pre_lo,
            "pre_hi": pre_hi, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window,
            "sinks": sinks}


def _append(name, dtype, seqs, lo, hi, pre_lo, pre_hi, kv_heads, dim, page):
    return {"name": name, "op": "append", "dtype": dtype, "seqs": seqs, "new_lo": lo, "new_hi": hi, "pre_lo": pre_lo,
            "pre_hi": pre_hi, "kv_heads": kv_heads, "dim": dim, "page": page}


def _copy(name, dtype, layers, pages, count, kv_heads, dim, page):
    return {"name": name, "op": "copy", "dtype": dtype, "layers": layers, "pages": pages, "count": count,
            "kv_heads": kv_heads, "dim": dim, "page": page}


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    dtype = rng.choice(("fp16", "bf16"))
    dim = rng.choice((64, 96, 128, 128, 128, 256))
    page = rng.choice((16, 32, 64, 128))
    q_heads, kv_heads = rng.choice(((32, 32), (32, 8), (32, 4), (64, 8), (28, 4), (12, 12), (20, 1)))
    window = rng.choice((0, 0, log_int(16, 8192)))
    sinks = rng.choice((0, 1, 4, 64)) if window else 0
    op = rng.choice(("decode", "decode", "prefill", "prefill", "append", "copy"))
    if op == "decode":
        seqs = log_int(1, 128)
        hi = log_int(1, max(1, min(131072, (1 << 31) // (seqs * kv_heads * dim * 4))))
        case = _decode("", dtype, seqs, rng.randint(1, hi), hi, q_heads, kv_heads, dim, page, window, sinks)
    elif op == "prefill":
        seqs = log_int(1, 16)
        # Query rows x keys, over all heads, up to a 4096-token prompt of 32 heads of 128.
        most = (1 << 24) * 32 * 128 // (q_heads * dim * seqs)
        pre = rng.choice((0, 0, log_int(1, 24576)))
        hi = log_int(1, min(6000, int(math.sqrt(most + pre * pre / 4.0) - pre / 2.0)))
        case = _prefill("", dtype, seqs, rng.randint(1, hi), hi, rng.randint(0, pre), pre, q_heads, kv_heads, dim, page,
                        window, sinks)
    elif op == "append":
        seqs = log_int(1, 128)
        hi = log_int(1, max(1, 16384 // seqs))
        pre = log_int(1, 4096)
        case = _append("", dtype, seqs, rng.randint(1, hi), hi, rng.randint(0, pre), pre, kv_heads, dim, page)
    else:
        layers = log_int(1, 40)
        most = (400 << 20) // (layers * kv_heads * dim * page * 2)      # bytes of the copied keys
        count = log_int(1, max(1, min(400, most)))
        case = _copy("", dtype, layers, 2 * count + rng.randint(0, 16), count, kv_heads, dim, page)
    del case["name"]
    return case


def _lens(lo, hi, count):
    """``count`` lengths from lo to hi, both ends among them where count > 1."""
    if count == 1:
        return [hi]
    return [lo, hi] + [lo + int((hi - lo) * math.modf(0.6180339887498949 * (i + 1))[0]) for i in range(count - 2)]


def _rows(case):
    """(new tokens, cached tokens with the new ones) of every sequence."""
    if case["op"] == "decode":
        lens = _lens(case["len_lo"], case["len_hi"], case["seqs"])
        return [1] * len(lens), lens
    new = _lens(case["new_lo"], case["new_hi"], case["seqs"])
    pre = _lens(case["pre_lo"], case["pre_hi"], case["seqs"])[::-1]
    return new, [n + p for n, p in zip(new, pre)]


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    if case["op"] == "copy":
        shape = (case["layers"], case["pages"], heads, page, dim)
        order = torch.randperm(case["pages"], generator=gen, device=dev).to(torch.int32)
        return {"case": case, "k": normal(*shape), "v": normal(*shape), "src": order[:case["count"]].contiguous(),
                "dst": order[case["count"]:2 * case["count"]].contiguous()}

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
    state = {
        "case": case, "k": normal(pages, heads, page, dim), "v": normal(pages, heads, page, dim), "table": table,
        "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
        "starts": torch.tensor(starts, dtype=torch.int32, device=dev),
        "tokens": starts[-1], "max_len": max(lens), "max_new": max(new),
    }
    if case["op"] == "append":
        state["new_k"], state["new_v"] = normal(starts[-1], heads, dim), normal(starts[-1], heads, dim)
        return state
    state["q"] = normal(starts[-1], case["q_heads"], dim)
    state["scale"] = 1.0 / math.sqrt(dim)
    # What a serving program allocates once for its batch.
    state["out"] = torch.empty_like(state["q"])
    state["ws"] = {}
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import sparse_int4_gemm_amd as slim

    case = s["case"]
    if case["op"] == "copy":
        slim.kv_copy_pages(s["k"], s["v"], s["src"], s["dst"])
        return [s["k"], s["v"]]
    if case["op"] == "append":
        slim.kv_append(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["lens"], s["starts"])
        return [s["k"], s["v"]]
    if not s["ws"]:
        s["ws"]["ws"] = slim.workspace_attention(s["tokens"], case["seqs"], case["q_heads"], case["kv_heads"],
                                                 case["dim"])
    if case["op"] == "decode":
        return slim.attention_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], max_len=s["max_len"],
                                     window=case["window"], sinks=case["sinks"], scale=s["scale"], ws=s["ws"]["ws"],
                                     out=s["out"])
    return slim.attention_prefill(s["q"], s["k"], s["v"], s["table"], s["lens"], s["starts"], max_len=s["max_len"],
                                  window=case["window"], sinks=case["sinks"], scale=s["scale"], ws=s["ws"]["ws"],
                                  out=s["out"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "copy":
        src, dst = s["src"].long(), s["dst"].long()
        s["k"][:, dst] = s["k"][:, src]
        s["v"][:, dst] = s["v"][:, src]
        return [s["k"], s["v"]]
    # Sequence and position of every token, then the place of that position in the pool.
    starts, lens, page = s["starts"].long(), s["lens"].long(), case["page"]
    token = torch.arange(s["tokens"], device=starts.device)
    seq = (token[:, None] >= starts[None, 1:]).sum(1)
    row = token - starts[seq]
    pos = lens[seq] - (starts[seq + 1] - starts[seq]) + row
    if case["op"] == "append":
        at = s["table"].long()[seq, pos // page]
        s["k"][at, :, pos % page] = s["new_k"]
        s["v"][at, :, pos % page] = s["new_v"]
        return [s["k"], s["v"]]
    return _attention_plain(s, seq, row, pos)


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
    k = s["k"][table].float().transpose(1, 2).reshape(seqs, heads, -1, dim)
    v = s["v"][table].float().transpose(1, 2).reshape(seqs, heads, -1, dim)
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
    row = case["kv_heads"] * case["dim"] * size
    if case["op"] == "copy":
        return {"bytes": 4 * case["layers"] * case["count"] * case["page"] * row + 8 * case["count"], "flops": 0}
    new, lens = _rows(case)
    tokens = sum(new)
    small = 4 * (2 * len(lens) + 1) + 4 * sum(-(-n // case["page"]) for n in lens)
    if case["op"] == "append":
        return {"bytes": 4 * tokens * row + small, "flops": 0}
    pairs = keys = 0
    for n, length in zip(new, lens):
        a, b = _span(length - n, length, case["window"], case["sinks"])
        pairs, keys = pairs + a, keys + b
    q_row = case["q_heads"] * case["dim"]
    return {"bytes": 2 * keys * row + 2 * tokens * q_row * size + small, "flops": 4 * pairs * q_row}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        k, v = s["k"].clone(), s["v"].clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            k[:, b], v[:, b] = s["k"][:, a], s["v"][:, a]
        return [k.double(), v.double()]
    new, lens = _rows(case)
    table, page = s["table"].tolist(), case["page"]
    if case["op"] == "append":
        at = 0
        k, v = s["k"], s["v"]
        for b, (n, length) in enumerate(zip(new, lens)):
            i = 0
            while i < n:                                 # as much as the page of this position takes
                pos = length - n + i
                take = min(n - i, page - pos % page)
                for pool, rows in ((k, s["new_k"]), (v, s["new_v"])):
                    pool[table[b][pos // page], :, pos % page:pos % page + take] = rows[at + i:at + i + take].transpose(0, 1)
                i += take
            at += n
        return [k.double(), v.double()]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    share, at = case["q_heads"] // case["kv_heads"], 0
    for b, (n, length) in enumerate(zip(new, lens)):
        ids = s["table"][b, :-(-length // page)].long()
        i = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hide = j > i
        if case["window"]:
            hide = hide | ((i - j >= case["window"]) & (j >= case["sinks"]))
        for h in range(case["kv_heads"]):
            k = s["k"][ids, h].reshape(-1, case["dim"])[:length].double()
            v = s["v"][ids, h].reshape(-1, case["dim"])[:length].double()
            for g in range(h * share, (h + 1) * share):
                a = (s["q"][at:at + n, g].double() @ k.t()) * s["scale"]
                a = torch.softmax(a.masked_fill(hide, -math.inf), dim=1)
                out[at:at + n, g] = a @ v
        at += n
    return out

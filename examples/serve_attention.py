"""The attention half of a decoder block served with this library: compressed
q/k/v/o projections (slim.linear), rotary positions on the way to a paged
key-value cache (slim.kv_append_rope, slim.KVCache), attention of the prompts
(slim.attention_prefill) and of single tokens (slim.attention_decode); with
--cache-bits 4 the same over a cache of 4 bits a value.

Prompts of different lengths are prefilled together, one conversation is
forked, all of them decode some tokens, one ends, the cache is compacted and the
rest go on.  Weights and inputs are random; the last outputs are compared with
plain float32 attention over the cached keys and values.

  python examples/serve_attention.py [--hidden 4096] [--kv-heads 32] [--steps 32] [--window 0] [--cache-bits 16]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_int4_gemm_amd as slim  # noqa: E402

HEAD_DIM = 128


class Projection:
    """A compressed weight [N, K] with a rank-r adapter, and its workspaces."""

    def __init__(self, gen, N, K, rank):
        std = K ** -0.5
        self.w = slim.pack(torch.randn((N, K), generator=gen, device="cuda") * std)
        self.lt = (torch.randn((rank, K), generator=gen, device="cuda") * std).half()
        self.rt = (torch.randn((N, rank), generator=gen, device="cuda") * 0.1 * rank ** -0.5).half()
        self.ws = {}

    def __call__(self, x):
        m = x.shape[0]
        if m not in self.ws:
            self.ws[m] = slim.workspace(m, self.w.N, self.w.K, self.lt.shape[0])
        return slim.linear(x, self.w, self.lt, self.rt, ws=self.ws[m])


class AttentionBlock:
    def __init__(self, hidden, kv_heads, pages, page_size, window, sinks, cache_bits=16, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.q_heads, self.kv_heads = hidden // HEAD_DIM, kv_heads
        self.window, self.sinks = window, sinks
        rank = max(32, hidden // 10 // 32 * 32)
        self.q, self.k, self.v = (Projection(gen, n * HEAD_DIM, hidden, rank) for n in (self.q_heads, kv_heads, kv_heads))
        self.o = Projection(gen, hidden, hidden, rank)
        self.cache = slim.KVCache(1, pages, kv_heads, HEAD_DIM, page_size=page_size, bits=cache_bits)
        self.rope = slim.Rope(HEAD_DIM)
        self.ws = slim.workspace_attention(1, 1, self.q_heads, kv_heads, HEAD_DIM)     # serves every batch of these heads

    def step(self, x, seqs, counts):
        """x [tokens, hidden]: counts[i] new tokens of seqs[i].  Returns the block's
        output, the turned queries and the attention's output (for the check)."""
        if self.window:                   # (only now: the tokens of the step before saw these pages)
            for s in seqs:
                self.cache.drop(s, self.window, self.sinks)
        batch = self.cache.extend(seqs, counts)
        q = self.q(x).view(-1, self.q_heads, HEAD_DIM)
        k = self.k(x).view(-1, self.kv_heads, HEAD_DIM)
        v = self.v(x).view(-1, self.kv_heads, HEAD_DIM)
        pools = (self.cache.k[0], self.cache.v[0])
        if self.cache.bits == 4:
            append, decode, prefill = slim.kv_append_q4, slim.attention_decode_q4, slim.attention_prefill_q4
        else:
            append, decode, prefill = slim.kv_append_rope, slim.attention_decode, slim.attention_prefill
        append(k, v, *pools, batch.table, batch.lens, rope=self.rope, starts=batch.starts, q=q, q_out=q)
        kw = dict(max_len=batch.max_len, window=self.window, sinks=self.sinks, ws=self.ws)
        if all(c == 1 for c in counts):
            y = decode(q, *pools, batch.table, batch.lens, **kw)
        else:
            y = prefill(q, *pools, batch.table, batch.lens, batch.starts, **kw)
        return self.o(y.reshape(x.shape[0], -1)), q, y

    def plain(self, q, seq):
        """float32 attention of one sequence's last query over its cached keys."""
        n, size, pages = self.cache.length(seq), self.cache.page_size, self.cache.pages(seq)
        j = torch.arange(n, device="cuda")
        seen = (j > n - 1 - self.window) | (j < self.sinks) if self.window else j >= 0
        j = j[seen]
        if self.cache.bits == 4:
            ints = torch.tensor([*pages, n, 0, n], dtype=torch.int32, device="cuda")
            k, v = slim.kv_read_q4(self.cache.k[0], self.cache.v[0], ints[None, :-3], ints[-3:-2], ints[-2:], n)
            k, v = k[j], v[j]
        else:
            page = torch.tensor(pages, device="cuda")[j // size]
            k, v = (pool[0][page, :, j % size] for pool in (self.cache.k, self.cache.v))
        k, v = (x.float().repeat_interleave(self.q_heads // self.kv_heads, 1) for x in (k, v))
        s = (k * q.float()).sum(-1) * HEAD_DIM ** -0.5
        w = torch.exp(s - s.amax(0))
        return (w[..., None] * v).sum(0) / w.sum(0)[:, None]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--kv-heads", type=int, default=32)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--cache-bits", type=int, choices=(4, 16), default=16)
    a = ap.parse_args(argv)
    prompts = [700, 33, 256]
    block = AttentionBlock(a.hidden, a.kv_heads, 200, 64, a.window, 4 if a.window else 0, a.cache_bits)
    cache = block.cache
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def tokens(n):
        return torch.randn((n, a.hidden), generator=gen, device="cuda").half()

    worst = 0.0

    def check(q, y, seqs):
        nonlocal worst
        for i, s in enumerate(seqs):
            want = block.plain(q[i], s)
            off = float((y[i].float() - want).norm() / want.norm())
            worst = max(worst, off if off == off else float("inf"))

    seqs = [cache.add() for _ in prompts]
    block.step(tokens(sum(prompts)), seqs, prompts)
    seqs.append(cache.fork(seqs[0]))                     # shares pages until one of the two writes
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.steps):
        _, q, y = block.step(tokens(len(seqs)), seqs, [1] * len(seqs))
    torch.cuda.synchronize()
    per_step = (time.perf_counter() - began) / max(a.steps, 1)
    if a.steps:
        check(q, y, seqs)
    cache.free(seqs.pop(0))
    moved = cache.compact()
    _, q, y = block.step(tokens(len(seqs)), seqs, [1] * len(seqs))
    check(q, y, seqs)
    print(f"{len(prompts)} prompts of {prompts} tokens, {a.steps} steps of {len(seqs) + 1} sequences: "
          f"{per_step * 1e6:.0f} us a step; compaction moved {moved} pages, {cache.free_pages} free; "
          f"largest relative error against float32 {worst:.1e}")
    return worst


if __name__ == "__main__":
    sys.exit(0 if main() < 2e-3 else 1)

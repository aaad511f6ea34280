"""The attention half of a decoder block served with this library: compressed
q/k/v/o projections (slim.linear), a paged key-value cache (slim.KVCache),
attention of the prompts (slim.attention_prefill) and of single tokens
(slim.attention_decode).

Prompts of different lengths are prefilled together, one conversation is
forked, all of them decode some tokens, one ends, the cache is compacted and the
rest go on.  Weights and inputs are random; the last outputs are compared with
plain float32 attention over the cached keys and values.

  python examples/serve_attention.py [--hidden 4096] [--kv-heads 32] [--steps 32] [--window 0]
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


def rotate(x, positions, base=10000.0):
    """Rotary positions on [tokens, heads, HEAD_DIM] (first and second half of a head paired)."""
    half = HEAD_DIM // 2
    freq = base ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = positions.float()[:, None, None] * freq
    a, b = x.float()[..., :half], x.float()[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1).to(x.dtype)


class AttentionBlock:
    def __init__(self, hidden, kv_heads, pages, page_size, window, sinks, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.q_heads, self.kv_heads = hidden // HEAD_DIM, kv_heads
        self.window, self.sinks = window, sinks
        rank = max(32, hidden // 10 // 32 * 32)
        self.q, self.k, self.v = (Projection(gen, n * HEAD_DIM, hidden, rank) for n in (self.q_heads, kv_heads, kv_heads))
        self.o = Projection(gen, hidden, hidden, rank)
        self.cache = slim.KVCache(1, pages, kv_heads, HEAD_DIM, page_size=page_size)
        self.ws = slim.workspace_attention(1, 1, self.q_heads, kv_heads, HEAD_DIM)     # serves every batch of these heads

    def step(self, x, seqs, counts):
        """x [tokens, hidden]: counts[i] new tokens of seqs[i].  Returns the block's
        output, the queries and the attention's output (for the check)."""
        if self.window:                   # (only now: the tokens of the step before saw these pages)
            for s in seqs:
                self.cache.drop(s, self.window, self.sinks)
        batch = self.cache.extend(seqs, counts)
        at = [p for s, c in zip(seqs, counts) for p in range(self.cache.length(s) - c, self.cache.length(s))]
        positions = torch.tensor(at, device=x.device)
        q = rotate(self.q(x).view(-1, self.q_heads, HEAD_DIM), positions)
        k = rotate(self.k(x).view(-1, self.kv_heads, HEAD_DIM), positions)
        v = self.v(x).view(-1, self.kv_heads, HEAD_DIM)
        pools = (self.cache.k[0], self.cache.v[0])
        slim.kv_append(k, v, *pools, batch.table, batch.lens, batch.starts)
        kw = dict(max_len=batch.max_len, window=self.window, sinks=self.sinks, ws=self.ws)
        if all(c == 1 for c in counts):
            y = slim.attention_decode(q, *pools, batch.table, batch.lens, **kw)
        else:
            y = slim.attention_prefill(q, *pools, batch.table, batch.lens, batch.starts, **kw)
        return self.o(y.reshape(x.shape[0], -1)), q, y

    def plain(self, q, seq):
        """float32 attention of one sequence's last query over its cached keys."""
        n, size, pages = self.cache.length(seq), self.cache.page_size, self.cache.pages(seq)
        j = torch.arange(n, device="cuda")
        seen = (j > n - 1 - self.window) | (j < self.sinks) if self.window else j >= 0
        j = j[seen]
        page = torch.tensor(pages, device="cuda")[j // size]
        share = self.q_heads // self.kv_heads
        k, v = (pool[0][page, :, j % size].float().repeat_interleave(share, 1) for pool in (self.cache.k, self.cache.v))
        s = (k * q.float()).sum(-1) * HEAD_DIM ** -0.5
        w = torch.exp(s - s.amax(0))
        return (w[..., None] * v).sum(0) / w.sum(0)[:, None]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--kv-heads", type=int, default=32)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args(argv)
    prompts = [700, 33, 256]
    block = AttentionBlock(a.hidden, a.kv_heads, 200, 64, a.window, 4 if a.window else 0)
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

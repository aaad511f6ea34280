"""Plain NumPy fp64 statement of the paged cache and the attention over it
(contract: include/slim.h).  Nothing here is shared with the HIP kernels."""
from __future__ import annotations

import numpy as np


def visible(p: int, keys: int, window: int, sinks: int) -> np.ndarray:
    """Which of keys 0 .. keys - 1 a query at position p sees."""
    j = np.arange(keys)
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attention(q, kpool, vpool, table, lens, starts, scale, window=0, sinks=0):
    """q [tokens, q_heads, dim], pools [pages, kv_heads, page, dim], table
    [seqs, width], lens [seqs], starts [seqs + 1] or None.  Returns (out,
    lse, mass): fp64 outputs, the log of the softmax sums, and the softmax
    weighted mean of |v|, which scales every rounding error of an output."""
    q, kpool, vpool = (np.asarray(x, dtype=np.float64) for x in (q, kpool, vpool))
    tokens, q_heads, dim = q.shape
    pages, kv_heads, page, _ = kpool.shape
    share = q_heads // kv_heads
    seqs = len(lens)
    starts = np.arange(seqs + 1) if starts is None else np.asarray(starts)
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((tokens, q_heads), -np.inf)
    for b in range(seqs):
        rows = range(int(starts[b]), int(starts[b + 1]))
        n = max(int(lens[b]), 0)
        keys = min(n, table.shape[1] * page)
        if len(rows) == 0 or keys == 0:
            continue
        at = np.repeat(np.asarray(table[b], dtype=np.int64), page)[:keys]
        owned = (at >= 0) & (at < pages)
        slot = np.arange(keys) % page
        for i, t in enumerate(rows):
            seen = visible(n - len(rows) + i, keys, window, sinks) & owned
            if not seen.any():
                continue
            k, v = kpool[at[seen], :, slot[seen]], vpool[at[seen], :, slot[seen]]     # [keys, heads, dim]
            for h in range(q_heads):
                s = (k[:, h // share] @ q[t, h]) * scale
                m = s.max()
                w = np.exp(s - m)
                out[t, h] = w @ v[:, h // share] / w.sum()
                mass[t, h] = w @ np.abs(v[:, h // share]) / w.sum()
                lse[t, h] = m + np.log(w.sum())
    return out, lse, mass


def append(k_new, v_new, kpool, vpool, table, lens, starts):
    """The pools after the new rows were written (copies)."""
    kpool, vpool = kpool.copy(), vpool.copy()
    pages, _, page, _ = kpool.shape
    starts = np.arange(len(lens) + 1) if starts is None else starts
    for b in range(len(lens)):
        n = int(starts[b + 1]) - int(starts[b])
        for i in range(n):
            p = max(int(lens[b]), 0) - n + i
            if p < 0 or p // page >= table.shape[1]:
                continue
            at = int(table[b][p // page])
            if 0 <= at < pages:
                kpool[at, :, p % page] = k_new[int(starts[b]) + i]
                vpool[at, :, p % page] = v_new[int(starts[b]) + i]
    return kpool, vpool


def copy_pages(pool, src, dst):
    """pool [layers, pages, ...] after the copies (a copy)."""
    out = pool.copy()
    for a, b in zip(src, dst):
        if 0 <= a < pool.shape[1] and 0 <= b < pool.shape[1]:
            out[:, b] = pool[:, a]
    return out

"""Plain NumPy statement of the 4-bit key-value cache (contract:
include/slim.h).  Nothing here is shared with the HIP kernels."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
RANGE = {"fp16": (-23, 13), "bf16": (-125, 125)}


def encode(x, dtype):
    """Codes (uint8, x's shape) and scale bytes [..., dim / 32] of x [..., dim]."""
    x = np.asarray(x, dtype=np.float64)
    groups = x.reshape(*x.shape[:-1], -1, 32)
    finite = np.isfinite(groups).all(-1)
    groups = np.where(finite[..., None], groups, 0.0)
    lo, hi = RANGE[dtype]
    limits = 7.0 * 2.0 ** np.arange(lo, hi + 1, dtype=np.float64)
    e = lo + np.minimum(np.searchsorted(limits, np.abs(groups).max(-1), side="left"), hi - lo)
    a = np.abs(groups) / 2.0 ** e[..., None].astype(np.float64)
    # The nearest level: that of code k + 1 from the middle between it and k's
    # on, the middle itself to the even code.
    code = np.zeros(groups.shape, dtype=np.uint8)
    for k in range(7):
        middle = (LEVELS[k] + LEVELS[k + 1]) / 2
        code += a >= middle if k % 2 else a > middle
    code |= np.signbit(groups).astype(np.uint8) << 3
    code = np.where(finite[..., None], code, 0).astype(np.uint8)
    return code.reshape(x.shape), np.where(finite, e + 127, 255).astype(np.uint8)


def decode(code, scale):
    """fp64 values of codes [..., dim] and scale bytes [..., dim / 32]."""
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    by = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127.0))
    return (v.reshape(*code.shape[:-1], -1, 32) * by[..., None]).reshape(code.shape)


def pack(code, scale):
    """The pool uint8 [pages, heads, page, dim * 17 / 32] of codes [pages, heads, page, dim] and scales [..., dim / 32]."""
    pages, heads, page, dim = code.shape
    codes = (code[..., 0::2] | code[..., 1::2] << 4).reshape(pages, -1)
    scales = scale.reshape(pages, heads, page // 16, 16, dim // 32).swapaxes(3, 4).reshape(pages, -1)
    return np.concatenate([codes, scales], 1).reshape(pages, heads, page, dim * 17 // 32)


def unpack(pool):
    """(codes, scales) of a pool."""
    pages, heads, page, row = pool.shape
    dim = row * 32 // 17
    flat, n = pool.reshape(pages, -1), heads * page * dim // 2
    codes = flat[:, :n].reshape(pages, heads, page, dim // 2)
    scales = flat[:, n:].reshape(pages, heads, page // 16, dim // 32, 16).swapaxes(3, 4).reshape(pages, heads, page, dim // 32)
    code = np.stack([codes & 15, codes >> 4], -1).reshape(pages, heads, page, dim)
    return code, scales


def append(k_new, v_new, kpool, vpool, table, lens, starts, dtype):
    """The pools after the new rows were written (copies)."""
    out = []
    pages, _, page, _ = kpool.shape
    starts = np.arange(len(lens) + 1) if starts is None else starts
    for pool, new in ((kpool, k_new), (vpool, v_new)):
        code, scale = (x.copy() for x in unpack(pool))
        new_code, new_scale = encode(new, dtype)
        for b in range(len(lens)):
            n = int(starts[b + 1]) - int(starts[b])
            for i in range(n):
                t, p = int(starts[b]) + i, max(int(lens[b]), 0) - n + i
                if not 0 <= t < len(new) or p < 0 or p // page >= table.shape[1]:
                    continue
                at = int(table[b][p // page])
                if 0 <= at < pages:
                    code[at, :, p % page] = new_code[t]
                    scale[at, :, p % page] = new_scale[t]
        out.append(pack(code, scale))
    return out

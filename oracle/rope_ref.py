"""Plain NumPy fp64 statement of the rotary positions (contract:
include/slim.h).  Nothing here is shared with the HIP kernels."""
from __future__ import annotations

import numpy as np


def turn(x, positions, freqs, interleaved=False, magnitude=1.0):
    """x [tokens, heads, dim] turned: pairs as complex numbers times magnitude * exp(i * position * freq)."""
    x = np.asarray(x, dtype=np.float64)
    n = len(freqs)
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    angle = np.multiply.outer(np.asarray(positions, dtype=np.float64), np.asarray(freqs, dtype=np.float64))
    z = (a + 1j * b) * (magnitude * np.exp(1j * angle))[:, None, :]
    y = x.copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def partner(x, n, interleaved=False):
    """|other element of the pair| for every element (0 for those that are not turned)."""
    y = np.zeros_like(np.abs(x))
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = np.abs(x[..., 1:2 * n:2]), np.abs(x[..., 0:2 * n:2])
    else:
        y[..., :n], y[..., n:2 * n] = np.abs(x[..., n:2 * n]), np.abs(x[..., :n])
    return y

"""Rotary positions: the frequencies of a rotation, as rope, kv_append_rope and
kv_append_q4 take them.

Pair i of a head's first rot_dim elements turns by position * f_i radians, f_i =
base^(-2 i / rot_dim) unless scaled for contexts longer than a model was trained
on.  The frequencies are 64-bit: those of a position far out need them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib

SCALINGS = ("none", "linear", "ntk", "yarn")
_FP32_MAX = torch.finfo(torch.float32).max


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 0, turns: tuple[float, float] = (32.0, 1.0)) -> tuple[torch.Tensor, float]:
    """Frequencies (float64 [rot_dim / 2], on the host) and the magnitude that go with them.

    linear: positions divided by `factor`.  ntk: the base stretched so that
    the slowest pair turns `factor` times slower and the fastest as before.
    yarn: pairs that turn turns[0] times and more in original_len positions
    as before, those that turn turns[1] times or less `factor` times slower, a
    ramp over the pairs between; the magnitude is 0.1 ln(factor) + 1."""
    if rot_dim <= 0 or rot_dim % 8:
        raise ValueError(f"rot_dim must be a positive multiple of 8, not {rot_dim}")
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {SCALINGS}, not {scaling!r}")
    if not (base > 1.0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freqs = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return freqs / factor, 1.0
    if scaling != "yarn":
        return freqs, 1.0
    if original_len <= 0 or not turns[0] > turns[1] > 0:
        raise ValueError("yarn needs original_len > 0 and turns of two falling positive numbers")

    def pair_of(t):              # the pair, a real number, that turns t times in original_len positions
        return rot_dim * math.log(original_len / (2.0 * math.pi * t)) / (2.0 * math.log(base))

    low, high = max(math.floor(pair_of(turns[0])), 0), min(math.ceil(pair_of(turns[1])), rot_dim - 1)
    slow = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
    return freqs * (1.0 - slow) + freqs / factor * slow, 0.1 * math.log(factor) + 1.0


class Rope:
    """A rotation on the GPU, made once for a model.

    interleaved: pair i is elements 2 i and 2 i + 1 of a head, otherwise i and
    i + rot_dim / 2.  freqs: float64 [rot_dim / 2], in place of base and scaling;
    magnitude: in place of theirs.

    Its frequencies are made on the current stream, and calls read them when they run.  It
    may be let go after a call on any stream, but has to be kept as long as a
    graph that captured one is replayed."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_len: int = 0, turns: tuple[float, float] = (32.0, 1.0),
                 freqs: torch.Tensor | None = None, magnitude: float | None = None, device="cuda"):
        if freqs is None:
            freqs, own = rope_frequencies(rot_dim, base, scaling, factor, original_len, turns)
            magnitude = own if magnitude is None else magnitude
        elif rot_dim <= 0 or rot_dim % 8 or freqs.dtype != torch.float64 or freqs.shape != (rot_dim // 2,):
            raise ValueError(f"freqs must be float64 [rot_dim / 2] and rot_dim a multiple of 8, got {freqs.dtype} "
                             f"{tuple(freqs.shape)} for {rot_dim}")
        magnitude = 1.0 if magnitude is None else float(magnitude)
        if not abs(magnitude) <= _FP32_MAX:
            raise ValueError("magnitude must be finite and within fp32's range")
        self._freqs = freqs.to(device, copy=True).contiguous()
        self.made_on = _lib._current_stream(self._freqs.device) if self._freqs.is_cuda else None
        self.params = _lib.Rotation(ctypes.c_void_p(self._freqs.data_ptr()), rot_dim, int(bool(interleaved)), magnitude)

    # (None to be replaced: calls pass on `params`, and in it the frequencies' address.)
    @property
    def freqs(self) -> torch.Tensor:
        """The frequencies on the GPU."""
        return self._freqs

    @property
    def rot_dim(self) -> int:
        return self.params.rot_dim

    @property
    def interleaved(self) -> bool:
        return bool(self.params.interleaved)

    @property
    def magnitude(self) -> float:
        return self.params.magnitude

"""A rotation's magnitude is the 64-bit number that it was made with, down to the
kernels (of 4-bit keys it chooses codes: test_q4_borders_gpu.py); one that fp32, in
which halves are turned, cannot hold is refused."""
import ctypes
import math

import pytest

import sparse_int4_gemm_amd as slim
from sparse_int4_gemm_amd import _lib

P = 0x10000        # aligned, never dereferenced


@pytest.mark.parametrize("magnitude", [0.7, -1.0 - 2.0 ** -40, 0.1 * math.log(40.0) + 1.0, 3.4028234663852886e38])
def test_it_is_passed_on_whole(magnitude):
    rope = slim.Rope(8, magnitude=magnitude, device="cpu")
    assert rope.magnitude == rope.params.magnitude == magnitude


def test_yarns_is_its_own():
    rope = slim.Rope(64, scaling="yarn", factor=40.0, original_len=4096, device="cpu")
    assert rope.params.magnitude == slim.rope_frequencies(64, scaling="yarn", factor=40.0, original_len=4096)[1]


@pytest.mark.parametrize("magnitude", [3.41e38, -1e39, 1e308, float("inf"), float("nan")])
def test_it_must_fit_fp32(magnitude):
    with pytest.raises(ValueError):
        slim.Rope(8, magnitude=magnitude, device="cpu")
    bad = ctypes.byref(_lib.Rotation(P, 64, 0, magnitude))
    assert _lib.load().slim_rope(P, 512, P, 512, 1, 4, 128, 0, P, bad, None) == _lib.SLIM_EINVAL

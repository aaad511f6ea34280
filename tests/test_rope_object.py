"""A Rope owns the frequencies whose address its calls pass on."""
import pytest
import torch

import sparse_int4_gemm_amd as slim


def test_frequencies_are_its_own():
    freqs = torch.arange(1, 5, dtype=torch.float64)
    rope = slim.Rope(8, freqs=freqs, device="cpu")
    assert rope.params.freqs == rope.freqs.data_ptr() != freqs.data_ptr()
    freqs.zero_()
    assert rope.freqs.tolist() == [1, 2, 3, 4]
    with pytest.raises(AttributeError):
        rope.freqs = freqs
    strided = slim.Rope(8, freqs=torch.arange(8, dtype=torch.float64)[::2], device="cpu")
    assert strided.freqs.is_contiguous() and strided.freqs.tolist() == [0, 2, 4, 6]

"""A Rope's attributes are those of the struct that its calls pass on: they cannot
be set to others beside it."""
import pytest

import sparse_int4_gemm_amd as slim


@pytest.mark.parametrize("name,value", [("rot_dim", 16), ("interleaved", True), ("magnitude", 2.0)])
def test_they_cannot_be_set(name, value):
    rope = slim.Rope(32, magnitude=0.5, device="cpu")
    before = getattr(rope, name)
    with pytest.raises(AttributeError):
        setattr(rope, name, value)
    assert getattr(rope, name) == before == getattr(rope.params, name)


def test_they_have_their_types():
    rope = slim.Rope(8, interleaved=1, magnitude=2, device="cpu")
    assert rope.interleaved is True and rope.rot_dim == 8 and rope.magnitude == 2.0 and isinstance(rope.magnitude, float)

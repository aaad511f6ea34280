"""What a refusal of a pool's type names: the types that the call takes."""
import types

import pytest
import torch

from sparse_int4_gemm_amd import _lib


def pool(dtype):
    """As much of a tensor on the GPU as the checks look at."""
    return types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0), shape=torch.Size((4, 2, 16, 64)), dtype=dtype)


def test_copies_name_pages_of_bytes_too():
    for bad in (torch.float32, torch.int8):
        with pytest.raises(TypeError, match="float16, bfloat16 or uint8"):
            _lib.slim_kv_copy_pages(pool(bad), pool(bad), None, None)


def test_other_calls_do_not():
    for bad in (torch.float32, torch.uint8):
        with pytest.raises(TypeError, match=r"float16 or bfloat16$"):
            _lib.slim_kv_append(None, None, pool(bad), pool(bad), None, None)

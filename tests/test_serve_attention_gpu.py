"""The serving example end to end at small sizes: compressed projections, cache,
prompt and single-token attention, fork, free, drop and compaction together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("argv", [["--hidden", "512", "--kv-heads", "4"], ["--hidden", "1024", "--kv-heads", "2", "--window", "100"],
                                  ["--hidden", "512", "--kv-heads", "1", "--steps", "0"]])
def test_serving_example(argv):
    spec = importlib.util.spec_from_file_location("serve_attention", os.path.join(ROOT, "examples", "serve_attention.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # Attention outputs are fp16: two roundings (weights or their split, output) of 2^-11, against float32.
    assert example.main(argv) < 2e-3

"""The serving example over a cache of 4 bits: append, prompt and single-token
attention, reading back, fork, free, drop and compaction together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("argv", [["--hidden", "512", "--kv-heads", "4"], ["--hidden", "1024", "--kv-heads", "2", "--window", "100"],
                                  ["--hidden", "512", "--kv-heads", "1", "--steps", "0"],
                                  ["--hidden", "512", "--kv-heads", "1", "--window", "64"]])
def test_serving_example(argv):
    spec = importlib.util.spec_from_file_location("serve_attention", os.path.join(ROOT, "examples", "serve_attention.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # Against float32 on the values that the codes stand for: two roundings of fp16, as over 16 bits.
    assert example.main([*argv, "--cache-bits", "4"]) < 2e-3

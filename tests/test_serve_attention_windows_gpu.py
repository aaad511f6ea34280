"""The serving example's own check: results that are no numbers fail it."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("serve_attention", os.path.join(ROOT, "examples", "serve_attention.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_result_that_is_no_number_fails(example, monkeypatch):
    plain = example.AttentionBlock.plain
    monkeypatch.setattr(example.AttentionBlock, "plain", lambda *a: plain(*a) * float("nan"))
    assert not example.main(["--hidden", "512", "--kv-heads", "1", "--steps", "1"]) < 2e-3

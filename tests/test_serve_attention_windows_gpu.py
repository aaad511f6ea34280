"""The serving example's own check at windows whose first key is the last one of a
page that the next token no longer sees, and what it makes of results that are no numbers."""
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


# After the steps the lengths are 732, 65, 288 and 732, then one more: of windows 29 to 93 (and 157) the
# first key of 732 is 703, of page 10's end; of 97 that of 288; of 94 that of 733.
@pytest.mark.parametrize("window", [29, 93, 157, 97, 94, 64, 1])
def test_every_window_passes_its_check(example, window):
    assert example.main(["--hidden", "512", "--kv-heads", "1", "--window", str(window)]) < 2e-3


def test_a_result_that_is_no_number_fails(example, monkeypatch):
    plain = example.AttentionBlock.plain
    monkeypatch.setattr(example.AttentionBlock, "plain", lambda *a: plain(*a) * float("nan"))
    assert not example.main(["--hidden", "512", "--kv-heads", "1", "--steps", "1"]) < 2e-3

"""What the example's loop answers or refuses before it touches a GPU."""
import importlib.util
import os
from types import SimpleNamespace

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def generate():
    spec = importlib.util.spec_from_file_location(
        "decode_loop_host", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.generate


def test_no_tokens_asked_for(generate):
    model = SimpleNamespace(num_pages=9, page_size=4)
    assert generate(model, [[1, 2], [3]], 0) == ([[], []], 9)
    assert generate(model, [], 5) == ([], 9)


def test_an_empty_prompt_is_refused(generate):
    with pytest.raises(ValueError, match="prompt 1"):
        generate(SimpleNamespace(num_pages=9, page_size=4), [[1], []], 3)

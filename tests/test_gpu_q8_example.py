"""The example that runs mapping, 8-bit writes, a prompt and decode steps together."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_on_mapped_cache():
    spec = importlib.util.spec_from_file_location("decode_on_mapped_cache",
                                                  os.path.join(ROOT, "examples", "decode_on_mapped_cache.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    r = example.run(tokens=1000, layers=3, heads=2, group=4, k=2, question=37, steps=5)
    # a code is off by at most 2^-4 of its value, keys and values alike
    assert 0 < r["error"] < 2 * 2.0 ** -4
    assert r["graph_is_eager"]
    assert r["bytes_8"] < 0.51 * r["bytes_16"]

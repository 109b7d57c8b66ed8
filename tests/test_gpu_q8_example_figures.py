"""What the example prints is what it says it is: the time of a step, and the attention's own error apart from the codes' rounding."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_on_mapped_cache",
                                                  os.path.join(ROOT, "examples", "decode_on_mapped_cache.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_attention_adds_a_rounding_of_the_output(example):
    """Over the values that the cache holds, the output is off by its own rounding, 2^-9 in the mean square at most, and by less than
    that again."""
    r = example.run(tokens=1000, layers=3, heads=2, group=4, k=2, question=37, steps=2)
    assert 0 < r["own_error"] < 2.0 ** -8 < r["error"]


def test_the_steps_time_is_the_steps(example, monkeypatch):
    """Drawing the inputs, made slow here, is not counted."""
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    cycles = 20000000
    torch.cuda._sleep(1000)
    begin.record()
    torch.cuda._sleep(cycles)
    end.record()
    torch.cuda.synchronize()
    slept_us = begin.elapsed_time(end) * 1e3
    assert slept_us > 3000
    draw = torch.Tensor.normal_

    def slow(self, *args, **kwargs):
        torch.cuda._sleep(cycles)
        return draw(self, *args, **kwargs)

    monkeypatch.setattr(torch.Tensor, "normal_", slow)
    r = example.run(tokens=300, layers=2, heads=2, group=4, k=2, question=20, steps=4)
    assert 0 < r["step_us"] < slept_us / 2

"""The serving example end to end: W8A8 projections around the 8-bit cache, ragged prompts, then graph-replayed steps."""
import importlib.util
import os

import pytest

from tests.gpu_util import say, torch_cuda

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_stays_near_the_unquantized_one():
    """8-bit rounding of a row of n normal values is a step of max / 127 with max about 4 sigma (n = 1024): an error of
    4 / 127 / sqrt(12) = 0.009 of the row.  Two layers quantize both operands and the cache quantizes keys and values: six
    such errors, at most 0.022 together (those of the keys act through the softmax).  The bound is twice that."""
    torch_cuda()
    spec = importlib.util.spec_from_file_location("w8a8_attention", os.path.join(ROOT, "examples", "w8a8_attention.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    diff, prompt_ms, step_us = example.serve(seqs=3, prompt=150, steps=12)
    say(f"  relative difference {diff:.4f}, prompts {prompt_ms:.2f} ms, step {step_us:.0f} us")
    assert 0.0 < diff < 0.044

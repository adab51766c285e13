"""The 4-bit decode loop of examples/rows4_decode.py, small: no status bit, and
the last output within bf16 rounding (half a step, 2^-8, of the largest value)
and f16 probabilities (2^-11) of attention over the unpacked rows."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_loop_over_4_bit_rows():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("rows4_decode", os.path.join(ROOT, "examples", "rows4_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    requests, layers, heads, steps = 3, 2, 5, 4
    error, status, weights = example.run(requests, layers, heads, tokens=900, k=70, hot=256, steps=steps)
    assert error <= 2.0 ** -8 + 2.0 ** -10
    assert not any(status)
    # every head spreads a weight of 1 a step
    total = weights.double().sum(2)
    assert torch.allclose(total, torch.full_like(total, heads * steps), rtol=1e-4)

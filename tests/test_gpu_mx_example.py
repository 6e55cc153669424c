"""The example that serves an attention layer in the microscaled 4-bit format.

Each stage against float32 on its own 4-bit operands: the bfloat16 output is
off by 2^-9 of an entry at most and the sums by far less, 2^-8 in all.  Against
the dense layer: 4-bit values are off by a quarter at most and by about a tenth
in the mean; inputs, weights, cache, attention's output and the last weight are
five such roundings, less than half together."""

import importlib.util
import os

import pytest

from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [dict(hidden=512, q_heads=8, heads=2, head_dim=64, batch=5, tokens=150, steps=4),
                                   dict(hidden=1024, q_heads=20, heads=1, head_dim=128, batch=33, tokens=70, steps=3),
                                   dict(hidden=768, q_heads=4, heads=4, head_dim=256, batch=1, tokens=900, steps=2)])
def test_a_layer_served_in_four_bits(sizes):
    announce(f"example layer {sizes}")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx_decode.py")
    spec = importlib.util.spec_from_file_location("mx_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors, us = example.run(timed=3, **sizes)
    assert us > 0
    for stage in ("projection", "attention", "output"):
        assert errors[stage] < 2.0 ** -8, errors
    assert errors["dense"] < 0.5, errors

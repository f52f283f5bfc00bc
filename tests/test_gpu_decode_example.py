"""The decode example runs all operators together: its error against the plain layer, and graph replays."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("four_bit,bound", [(False, 0.04), (True, 0.08)])
def test_decode_layer(four_bit, bound):
    """Each 8-bit rounding is off by 2.6% of its vector (a uniform error in a step of 2^-3 of its binade), independent over the
    elements, and an NVFP4 cache by about 10% of each value, averaged over the tokens of the softmax; the residual stream
    adds the two branches, each with its errors, to the exact input."""
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    print(f"[case] decode example, four_bit {four_bit}", flush=True)
    error, same, _, _ = m.run(steps=40, batch=3, four_bit=four_bit)
    assert same, "a replayed graph differs from the eager steps"
    assert error < bound, error

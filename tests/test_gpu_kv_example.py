"""The example of decoding with encoded weights and the 4-bit cache, end to end."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_with_cache():
    spec = importlib.util.spec_from_file_location("decode_with_cache", os.path.join(ROOT, "examples", "decode_with_cache.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    # every layer's attention output is rounded to BF16 on both sides (2^-9 of it) after sums
    # that differ in their last places: a flipped rounding is 2^-8 of an element, and the rows
    # keep their FP32 residual besides
    assert m.main() < 2.0 ** -8

"""The layer of linear attention under examples/, as a user runs it."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [{}, {"T": 33, "B": 1, "heads": 3, "kv_heads": 3, "size": 32, "steps": 1}], ids=str)
def test_layer_prompt_steps_and_gradients(gpu, sizes):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import linear_attention_layer
    finally:
        sys.path.pop(0)
    apart, off = linear_attention_layer.main(**sizes)
    # fp32 throughout, the projections' inputs to 2^-22: the two ways differ in the
    # order of sums over at most 200 tokens and 64 rows (2^-24 each), which the
    # norms and projections enlarge a few times
    assert apart < 1e-4
    # central differences at 1e-2: the third order's 1e-4 with its factors, and
    # the sums' rounding over 2e-2
    assert off < 1e-2

"""The layer of the gated delta rule under examples/, as a user runs it."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [{}, {"T": 33, "B": 1, "heads": 3, "key_heads": 3, "size": 32, "steps": 1},
                                   {"T": 450, "B": 1, "heads": 2, "key_heads": 1, "size": 96, "steps": 3}], ids=str)
def test_layer_prompt_steps_and_gradients(gpu, sizes):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import gated_delta_layer
    finally:
        sys.path.pop(0)
    apart, eighth, off = gated_delta_layer.main(**sizes)
    # fp32 throughout, the projections' inputs to 2^-22: the two ways differ in the
    # order of sums over at most 450 tokens and 96 rows (2^-24 each, added as
    # independent ones: 16 * 2^-24 * 25 = 2.4e-5), which the norm of a head and the last projection
    # carry on at about their size
    assert apart < 1e-4
    # one rounding to e4m3, and two of fp32 in the scaled value
    assert eighth < 1.001
    # central differences at 1e-2 of directions of 0.2: the third order's 1e-4 * 0.04 with its
    # factors, and the sums' rounding over 2e-2
    assert off < 1e-2

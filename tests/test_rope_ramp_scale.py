"""The factor of the rotated values that a ramp table comes with (no GPU)."""
import math

import numpy as np
import pytest

import paged_kv_attention_cache_gb300 as tl


@pytest.mark.parametrize("factor,want", [
    (1.0, 1.0), (0.5, 1.0), (1e-3, 1.0),
    (math.exp(-10), 1.0), (1e-6, 1.0),  # where 0.1 ln(factor) + 1 is 0 and below
    (1.25, 0.1 * math.log(1.25) + 1), (8.0, 0.1 * math.log(8.0) + 1), (40.0, 0.1 * math.log(40.0) + 1),
])
def test_positions_that_are_not_stretched_leave_the_values_alone(factor, want):
    _, scale = tl.tl_rope_freqs(64, 10000.0, tl.TL_ROPE_RAMP, factor=factor, trained_len=4096,
                                low=1.0, high=32.0, device="cpu")
    assert scale == float(np.float32(want))

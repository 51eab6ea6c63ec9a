"""Pins of the decode path's oracle where numbers end."""

import numpy as np

from oracle import decode as dec


def test_quantiser_holds_a_span_past_fp32_as_nan():
    top = float(np.finfo(np.float32).max)
    x = np.zeros((4, 64))
    x[0, :2] = 3e38, -3e38
    x[1, :2] = top, 0.0
    x[2, :2] = top / 2, -top / 2
    x[3, :2] = top, -2.0 ** 103      # rounds to 2^128
    _, s, z = dec.quantise(x)
    assert np.isnan(s[[0, 3]]).all() and np.isnan(z[[0, 3]]).all()
    assert np.isfinite(s[[1, 2]]).all() and np.isfinite(z[[1, 2]]).all()
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(x[3, 0]) - np.float32(x[3, 1])) and np.isinf(np.float32(x[0, 0]) - np.float32(x[0, 1]))

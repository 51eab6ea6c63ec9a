"""The rotary and decode calls where their ranges end, for both builds:
infinities and NaN beside rows that are settled in 64 bits, rows too large or
too small for fp32 squares, more tokens than a grid dimension holds, lengths
near 2^31, positions outside the tables, block tables much wider than the
requests. Bounds as in test_decode_gpu.py unless a test derives its own."""

import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from oracle import decode as dec
from test_decode_gpu import (DT, EPS, HALF, U, build_cache, check_attention, check_held, dev, f64, gen, numbers_of, randn,
                             random_cache, scales_of)

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


# ---------------------------------------------------------------------------
# Infinities, NaN and overflowing spans
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("embedded", [False, True])
@pytest.mark.parametrize("rest", [0.0, 0.25])
def test_a_group_that_is_not_finite_is_held_as_nan(kind, embedded, rest):
    # the other group of the row is constant: its step is 0, on a border
    # between two roundings, so the row's numbers are settled in 64 bits
    d, page = 128, 16
    bad = [{0: math.inf}, {5: -math.inf}, {63: math.nan}, {17: math.nan, 18: math.inf}, {8: 3e38, 40: -3e38}, {3: math.nan, 0: 1.0}]
    n = 2 * len(bad)
    v = torch.zeros(1, n, 1, d, dtype=DT[kind])
    want = torch.zeros(n, d, dtype=torch.bool)
    for i, entries in enumerate(bad):
        for j, at in ((2 * i, 0), (2 * i + 1, 64)):
            v[0, j, 0, 64 - at:128 - at] = rest
            for c, x in entries.items():
                v[0, j, 0, at + c] = x
            want[j, at:at + 64] = True
    cache = random_cache(1, 2, 1, page, d).to(dev())
    slot = torch.arange(n, device=dev()).view(1, n)
    kw = {}
    if embedded:
        kw = dict(ve=torch.zeros(3, d, dtype=DT[kind], device=dev()), tok=torch.ones(1, n, dtype=torch.int32, device=dev()))
    swa.kv4_append(cache, randn(1, 1, n, 1, d, dtype=DT[kind]).to(dev()), v.to(dev()), slot, **kw)
    kr, vr = (x[0, :, 0].cpu() for x in swa.kv4_read(cache, slot, dtype=torch.float32))
    assert torch.equal(torch.isnan(vr), want)
    assert torch.all(vr[~want] == rest) and torch.isfinite(kr).all()
    held = dec.dequantise(*dec.quantise(f64(v)[0, :, 0]))      # and the oracle says the same
    np.testing.assert_array_equal(np.isnan(held), want.numpy())

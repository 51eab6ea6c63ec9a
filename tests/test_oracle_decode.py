"""Pins of the float64 oracle of rotary tables and of the decode path against
closed forms, torch's own bf16 rounding, the training oracle, and worked
examples."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import decode as dec


def rng(seed):
    return np.random.default_rng(seed)


def test_bf16_rounding_is_torchs():
    x = np.concatenate([rng(0).standard_normal(4000) * 10.0 ** rng(1).integers(-30, 30, 4000),
                        [0.0, 1.0, -1.0, 1.00390625, 1.01171875, 3.39e38, 3.4e38, 1e-40, np.inf, -np.inf, np.nan]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(dec.bf16(x), want)


def test_tables_closed_forms():
    cos, sin = dec.rope_tables(5, 16)
    assert cos.shape == (5, 8) and np.all(cos[0] == 1) and np.all(sin[0] == 0)
    np.testing.assert_allclose(cos[:, 0], np.cos(np.arange(5)))              # theta_0 = 1
    np.testing.assert_allclose(dec.rope_frequencies(16, base=81.0)[4], 1 / 9.0)   # base^(-1/2)
    lin, far = dec.rope_tables(9, 32, scaling="linear", factor=4.0), dec.rope_tables(3, 32)
    np.testing.assert_allclose(lin[0][::4], far[0], atol=1e-15)              # positions interpolated
    ntk = dec.rope_frequencies(64, scaling="ntk", factor=8.0)
    plain = dec.rope_frequencies(64)
    assert ntk[0] == 1.0
    np.testing.assert_allclose(ntk[-1], plain[-1] / 8.0)    # the lowest frequency is stretched by the factor exactly
    parts = dec.rope_frequencies(64, scaling="by_parts", factor=8.0, orig_len=2048)
    turns = 2048 * plain / (2 * math.pi)
    np.testing.assert_allclose(parts[turns >= 32], plain[turns >= 32])
    np.testing.assert_allclose(parts[turns <= 1], plain[turns <= 1] / 8.0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(parts[mid] < plain[mid]) and np.all(parts[mid] > plain[mid] / 8)


def test_rotation_is_the_training_oracles_and_orthogonal():
    x = rng(2).standard_normal((7, 3, 16))
    cos, sin = dec.rope_tables(7, 16)
    want = oracle.rotary(x[None], cos, sin)[0]
    np.testing.assert_allclose(dec.rotate(x, cos, sin), want, atol=1e-14)
    np.testing.assert_allclose(dec.rotate(dec.rotate(x, cos, sin), cos, sin, inverse=True), x, atol=1e-14)
    # the interleaved layout is the split-half one under a permutation of channels
    perm = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    np.testing.assert_allclose(dec.rotate(x, cos, sin, interleaved=True)[..., perm], dec.rotate(x[..., perm], cos, sin),
                               atol=1e-14)
    part = dec.rotate(x, cos[:, :4], sin[:, :4])
    np.testing.assert_array_equal(part[..., 8:], x[..., 8:])
    # <g, R x> = <R^T g, x>
    g = rng(3).standard_normal(x.shape)
    for inter in (False, True):
        a = np.sum(g * dec.rotate(x, cos, sin, inter))
        b = np.sum(dec.rotate(g, cos, sin, inter, inverse=True) * x)
        assert abs(a - b) < 1e-12


def test_quantiser():
    x = rng(4).standard_normal((5, 128))
    x[1, :64] = 3.5              # a constant group
    x[2, 7] = np.nan
    x[3, 100] = np.inf
    n, s, z = dec.quantise(x)
    y = dec.dequantise(n, s, z)
    assert n.min() >= 0 and n.max() <= 15
    ok = ~np.isnan(np.repeat(s, 64, axis=-1).reshape(x.shape))
    assert np.isnan(y[2, :64]).all() and np.isnan(y[3, 64:]).all() and ok[2, 64:].all() and ok[3, :64].all()
    assert np.all(y[1, :64] == 3.5)
    # half a step, and what rounding s and z to bf16 moves the ends of the range by
    span = np.repeat(15 * s, 64, axis=-1).reshape(x.shape)
    zz = np.repeat(np.abs(z), 64, axis=-1).reshape(x.shape)
    assert np.all(np.abs(y - x)[ok] <= (span / 30 + span * 2.0 ** -8 + zz * 2.0 ** -8 + 1e-12)[ok])
    # borders go up
    row = np.zeros((1, 64))
    row[0, 0], row[0, 1], row[0, 2] = -8.0, 7.0, 0.5
    n, s, z = dec.quantise(row)
    assert s[0, 0] == 1.0 and z[0, 0] == 0.0 and n[0, 2] == 9 and n[0, 3] == 8


@pytest.mark.parametrize("d", [64, 128])
def test_cache_rows_come_back_and_neighbours_stay(d):
    r = rng(5)
    page, H = 32, 2
    cache = r.integers(0, 256, (3, H, page // 16, 18 * d)).astype(np.uint8)
    kp, vp = dec.nibble_places(d)
    assert sorted(kp) == list(range(d)) and sorted(np.concatenate([vp, vp + 4])) == list(range(2 * d))
    rows = {}
    for slot in (0, 1, 14, 15, 16, 37, 95):
        for h in range(H):
            k, v = r.standard_normal((2, d))
            kq, vq = dec.quantise(k[None]), dec.quantise(v[None])
            dec.write_row(cache, page, slot, h, [a[0] for a in kq], [a[0] for a in vq])
            rows[slot, h] = dec.dequantise(*kq)[0], dec.dequantise(*vq)[0]
    for (slot, h), (k, v) in rows.items():
        got = dec.read_row(cache, page, slot, h)
        np.testing.assert_array_equal(got[0], k)
        np.testing.assert_array_equal(got[1], v)


def test_attend_is_the_training_oracles_last_row():
    r = rng(6)
    T, Hq, Hkv, d = 40, 4, 2, 64
    q, k, v = r.standard_normal((1, T, Hq, d)), r.standard_normal((1, T, Hkv, d)), r.standard_normal((1, T, Hkv, d))
    gq, gk = 1 + 0.1 * r.standard_normal((2, d))
    cos, sin = dec.rope_tables(T, d)
    for window in (-1, 0, 7, 100):
        o, lse = oracle.attention_forward(q, k, v, gq, gk, window=window, eps=1e-6, rope=(cos, sin))
        kn = dec.rms_norm(dec.rotate(k[0], cos, sin), gk, 1e-6)
        got = dec.attend(q[0, -1], kn, v[0], window=window, gq=gq, cos=cos[-1], sin=sin[-1])
        np.testing.assert_allclose(got[0], o[0, -1], atol=1e-12)
        np.testing.assert_allclose(got[1], lse[0, :, -1], atol=1e-12)
    o, lse = dec.attend(q[0, 0], k[0][:0], v[0][:0])
    assert np.all(o == 0) and np.all(lse == -np.inf)


def test_plan_worked_example():
    # pages of 16: requests with 16, 5 and 0 tokens get 1, 12 and 20 more
    table = np.array([[7, -1, -1], [2, -1, -1], [-1, -1, -1]], np.int32)
    free = np.array([9, 4, 1, 3, 8], np.int32)
    p = dec.plan(np.array([16, 5, 0], np.int32), np.array([1, 12, 20], np.int32), table, free, 1, 16, 10, 36)
    assert p["table"].tolist() == [[7, 4, -1], [2, 1, -1], [3, 8, -1]]
    assert p["lens"].tolist() == [17, 17, 20] and p["cu"].tolist() == [0, 1, 13, 33]
    assert p["free_head"] == 5 and p["refused"] == 0
    assert p["slot"][0] == 4 * 16 and p["pos"][0] == 16
    assert p["slot"][1] == 2 * 16 + 5 and p["slot"][11] == 2 * 16 + 15 and p["slot"][12] == 16
    assert p["slot"][13] == 3 * 16 and p["slot"][32] == 8 * 16 + 3
    assert p["row"][33:].tolist() == [-1] * 3 and p["slot"][33:].tolist() == [-1] * 3
    # one page short: the last request is refused, a request that needs none behind it goes
    p = dec.plan(np.array([16, 0, 5], np.int32), np.array([1, 40, 2], np.int32), table[[0, 2, 1]], free, 3, 16, 10, 64)
    assert p["lens"].tolist() == [17, 0, 7] and p["free_head"] == 4 and p["refused"] == 1
    assert p["slot"][1:41].tolist() == [-1] * 40 and p["slot"][41] == 2 * 16 + 5

"""Pins of the oracle of the norm, the 4-bit weights and the drafted tokens
(oracle/serve.py): closed forms, differences, and other ways to the same numbers."""

import numpy as np
import pytest
import torch

from oracle import decode as dec
from oracle import serve


def rng(seed):
    return np.random.default_rng(seed)


def test_round8_is_the_nearest_of_all_numbers():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    codes = np.unique(codes[np.isfinite(codes)])
    x = np.concatenate([rng(0).uniform(-448, 448, 2000), rng(1).normal(size=2000) * 0.02, codes, [0.0]])
    y = serve.round8(x)
    assert np.all(np.isin(y, codes))
    assert np.all(np.abs(x - y) <= np.abs(x[:, None] - codes).min(1))
    assert np.array_equal(y, torch.tensor(x, dtype=torch.float64).float().to(torch.float8_e4m3fn).double().numpy())
    mid = (codes[1:] + codes[:-1]) / 2                # ties: the even one of the two
    even = torch.tensor(mid, dtype=torch.float64).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(serve.round8(mid), even)


def test_norm_is_torchs_and_its_8_bits_are_near():
    h, g = rng(2).normal(size=(5, 96)), 1 + 0.1 * rng(3).normal(size=96)
    y, rstd = serve.norm(h, g)
    want = torch.nn.functional.rms_norm(torch.tensor(h), (96,), torch.tensor(g), 1e-6).numpy()
    assert np.allclose(y, want, rtol=1e-12, atol=0)
    n, s = serve.norm8(h, g)
    assert np.abs(n).max(1).tolist() == [448.0] * 5
    assert np.all(np.abs(n * s[:, None] - y) <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * s[:, None])
    n0, s0 = serve.norm8(np.zeros((1, 96)))
    assert not n0.any() and not s0.any()


def test_norm_backward_by_differences():
    h, g = rng(4).normal(size=(3, 16)), 1 + 0.1 * rng(5).normal(size=16)
    dy, dh = rng(6).normal(size=(3, 16)), rng(7).normal(size=(3, 16))

    def loss(h, g):
        return (serve.norm(h, g)[0] * dy).sum() + (h * dh).sum()
    dx, dg = serve.norm_backward(h, serve.norm(h)[1], dy, g, dh)
    for a, grad in ((h, dx), (g, dg)):
        for i in np.ndindex(a.shape):
            e = np.zeros_like(a)
            e[i] = 1e-5
            up = loss(h + e, g) if a is h else loss(h, g + e)
            down = loss(h - e, g) if a is h else loss(h, g - e)
            assert abs((up - down) / 2e-5 - grad[i]) < 1e-7


@pytest.mark.parametrize("N,K", [(16, 64), (1, 8), (33, 200)])
def test_w4_numbers_are_near_and_the_bytes_hold_them(N, K):
    w = rng(8).normal(size=(N, K)).astype(np.float32).astype(np.float64)
    n, s = serve.w4_quantise(w)
    back = (n - 8) * np.repeat(s, 64, 1)[:, :K]
    # half a step, and where bf16 took the step down 7 steps fall short of the largest entry
    assert np.all(np.abs(back - w) <= (0.5 + 7 * 2.0 ** -8) * np.repeat(s, 64, 1)[:, :K])
    tiles = serve.w4_tiles(n, s)
    assert tiles.shape == (-(-N // 16), -(-K // 64), 544)
    assert np.array_equal(serve.w4_values(tiles, N, K), back)
    full = serve.w4_values(tiles, 16 * tiles.shape[0], 64 * tiles.shape[1])
    assert not full[N:].any() and not full[:, K:].any()


def test_w4_places_are_the_headers():
    # lane = 4 r + j, word w: e, q, hi = 0, 1 from the low nibble on
    seen = set()
    for r in range(8):
        for j in range(4):
            for w in range(4):
                for i in range(8):
                    e, q, hi = i // 4, i // 2 % 2, i % 2
                    byte, shift = serve.w4_place(r + 8 * hi, 16 * j + 4 * w + 2 * q + e)
                    assert (byte, shift) == (16 * (4 * r + j) + 4 * w + i // 2, 4 * (i % 2))
                    seen.add((byte, shift))
    assert len(seen) == 1024


def test_a_chain_of_drafted_tokens_is_as_many_decode_steps():
    n, ctx, Hq, Hkv, d = 4, 9, 4, 2, 64
    keys, vals, q = rng(9).normal(size=(ctx + n, Hkv, d)), rng(10).normal(size=(ctx + n, Hkv, d)), rng(11).normal(size=(n, Hq, d))
    cos, sin = dec.rope_tables(ctx + n, 32)
    pos, seen = serve.tree([-1, 0, 1, 2], ctx)
    assert pos == [9, 10, 11, 12] and seen == [1, 3, 7, 15]
    for window in (-1, 3):
        o, lse = serve.tree_attend(q, keys, vals, pos, seen, window, cos=cos, sin=sin)
        for i in range(n):
            ro, rl = dec.attend(q[i], keys[:ctx + i + 1], vals[:ctx + i + 1], window, cos=cos[ctx + i], sin=sin[ctx + i])
            assert np.allclose(o[i], ro, atol=1e-13) and np.allclose(lse[i], rl, atol=1e-13)


def test_tokens_see_their_own_branch_only():
    pos, seen = serve.tree([-1, 0, 0, 1, 2, -1], 5)
    assert pos == [5, 6, 6, 7, 7, 5]
    assert seen == [1, 0b11, 0b101, 0b1011, 0b10101, 0b100000]
    q, keys, vals = rng(12).normal(size=(6, 2, 64)), rng(13).normal(size=(11, 1, 64)), rng(14).normal(size=(11, 1, 64))
    o, lse = serve.tree_attend(q, keys, vals, pos, seen)
    for t in range(6):                          # what token t holds changes those that see it, and no other
        k2 = keys.copy()
        k2[5 + t] += 1
        o2, _ = serve.tree_attend(q, k2, vals, pos, seen)
        assert [bool(np.any(o2[i] != o[i])) for i in range(6)] == [bool(s >> t & 1) for s in seen]
    o0, l0 = serve.tree_attend(q, keys, vals, pos, [0] * 6)
    assert not o0.any() and np.all(l0 == -np.inf)


def test_the_measured_cases_hold_the_same_weights():
    from perf import more_operators as m
    w = torch.randint(0, 256, (3, 4, 544), dtype=torch.uint8, generator=torch.Generator().manual_seed(0))
    w[..., 512:].view(torch.bfloat16).copy_(torch.rand(3, 4, 16))
    want = serve.w4_values(w.numpy(), 37, 200)
    assert np.array_equal(m._weights(w, 37, 200).double().numpy(), want)

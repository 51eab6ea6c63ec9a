"""Float64 NumPy oracle of the norm with the residual's addition (8-bit output
and backward included), of projections with 4-bit weights, and of drafted tokens
over the decode path's cache. Plain definitions; imports nothing of the package.
"""

from __future__ import annotations

import math

import numpy as np

from .decode import bf16, rms_norm, rotate

TOP8 = 448.0


def round8(x):
    """|x| <= 448 to the nearest e4m3 number, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    e = np.maximum(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -9))), -6)
    unit = 2.0 ** (e - 3)
    return np.rint(x / unit) * unit


def norm(h, gain=None, eps=1e-6):
    """y, rstd of rows h [rows, C]."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * (1.0 if gain is None else gain), rstd


def norm8(h, gain=None, eps=1e-6):
    """The e4m3 numbers and the scales of rows h. The numbers come from u = gain h
    (products of at most 48 bits: exact here), where the rows' rstd has dropped out."""
    u = np.asarray(h, dtype=np.float64) * (1.0 if gain is None else gain)
    top = np.abs(u).max(-1)
    n = round8(u * TOP8 / np.where(top > 0, top, 1.0)[:, None])
    return n, top * norm(h, None, eps)[1] / TOP8


def norm_backward(h, rstd, dy, gain=None, dh=None):
    """dx, dgain."""
    xh = h * rstd[:, None]
    d = dy * (1.0 if gain is None else gain)
    dx = rstd[:, None] * (d - xh * (d * xh).mean(-1, keepdims=True))
    return dx + (0.0 if dh is None else dh), (dy * xh).sum(0)


def w4_quantise(w):
    """Numbers [N, K] (0..15) and steps [N, ceil(K / 64)] of weights w [N, K]."""
    w = np.asarray(w, dtype=np.float64)
    N, K = w.shape
    n = np.full((N, K), 8, dtype=np.int64)
    s = np.zeros((N, -(-K // 64)))
    for g in range(s.shape[1]):
        c = w[:, 64 * g:64 * g + 64]
        # the quotient in fp32, then bf16
        q = (np.abs(c).max(1).astype(np.float32) / np.float32(7.0)).astype(np.float64)
        s[:, g] = bf16(q)
        s[s[:, g] < 1e-36, g] = 0.0
        for i in range(N):
            st = s[i, g]
            if st == 0:
                continue
            k = np.clip(np.floor(c[i] / st + 8.5), 0, 15)
            # floor(w / s + 8.5) by its borders, whose products are exact here
            k -= (k > 0) & (c[i] < (k - 8.5) * st)
            k += (k < 15) & (c[i] >= (k - 7.5) * st)
            n[i, 64 * g:64 * g + 64] = k
    return n, s


def w4_place(row, col):
    """Byte of a tile and shift of the number of (row, column) within it, row < 16, col < 64."""
    lane = 4 * (row % 8) + col // 16
    nibble = 4 * (col % 2) + 2 * (col // 2 % 2) + row // 8
    return 16 * lane + 4 * (col % 16 // 4) + nibble // 2, 4 * (nibble % 2)


def w4_tiles(n, s):
    """The packed bytes of numbers and steps."""
    N, K = n.shape
    P, Q = -(-N // 16), -(-K // 64)
    full = np.full((16 * P, 64 * Q), 8, dtype=np.int64)
    full[:N, :K] = n
    steps = np.zeros((16 * P, Q))
    steps[:N] = s
    out = np.zeros((P, Q, 544), dtype=np.uint8)
    for r in range(16):
        for c in range(64):
            byte, shift = w4_place(r, c)
            out[:, :, byte] |= (full[r::16, c::64] << shift).astype(np.uint8)
        bits = (steps[r::16].astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
        at = 512 + 2 * (2 * (r % 8) + r // 8)
        out[:, :, at], out[:, :, at + 1] = bits & 255, bits >> 8
    return out


def w4_values(tiles, N, K):
    """The weights [N, K] that packed bytes stand for."""
    P, Q, _ = tiles.shape
    w = np.zeros((16 * P, 64 * Q))
    for r in range(16):
        at = 512 + 2 * (2 * (r % 8) + r // 8)
        bits = tiles[:, :, at].astype(np.uint32) | tiles[:, :, at + 1].astype(np.uint32) << 8
        step = (bits << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        for c in range(64):
            byte, shift = w4_place(r, c)
            w[r::16, c::64] = ((tiles[:, :, byte].astype(np.int64) >> shift & 15) - 8) * step
    return w[:N, :K]


def tree(parent, ctx):
    """Positions and visibility bits of one request's drafted tokens."""
    pos, seen = [], []
    for i, p in enumerate(parent):
        above = seen[p] if p >= 0 else 0
        seen.append(above | 1 << i)
        pos.append(ctx + bin(seen[i]).count("1") - 1)
    return pos, seen


def tree_attend(q, keys, values, pos, seen, window=-1, gq=None, eps=1e-6, scale=None, cos=None, sin=None, interleaved=False):
    """o [n, Hq, d], lse [n, Hq] of one request's n drafted tokens q [n, Hq, d], whose
    keys and values are the last n of [len, Hkv, d]; cos, sin: tables."""
    q = np.asarray(q, dtype=np.float64)
    n, Hq, d = q.shape
    ctx, G = len(keys) - n, Hq // keys.shape[1]
    if cos is not None:
        q = rotate(q, cos[list(pos)], sin[list(pos)], interleaved)
    q = rms_norm(q, gq, eps)
    scale = 1.0 / math.sqrt(d) if not scale else scale
    o, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf)
    for i in range(n):
        if seen[i] == 0:
            continue
        see = [j for j in range(ctx) if window < 0 or pos[i] - j <= window]
        see += [ctx + t for t in range(n) if seen[i] >> t & 1 and (window < 0 or pos[i] - pos[t] <= window)]
        for h in range(Hq if see else 0):
            z = scale * keys[see, h // G] @ q[i, h]
            p = np.exp(z - z.max())
            lse[i, h] = z.max() + np.log(p.sum())
            o[i, h] = p @ values[see, h // G] / p.sum()
    return o, lse

"""Float64 NumPy oracle of rotary tables and rotations, and of the decode path
(step plan, 4-bit paged cache, attention of one token per request). Plain
definitions, loops where they are clearest; imports nothing of the package.

bf16 rounding (the cache's scales) is done here on the float64 values.
"""

from __future__ import annotations

import math

import numpy as np

TILE = 16


def bf16(x):
    """float64 values rounded to the nearest bf16 (ties to even), as float64."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    fin = np.isfinite(x) & (x != 0.0)
    e = np.floor(np.log2(np.abs(x[fin])))
    e = np.maximum(e, -126)
    ulp = 2.0 ** (e - 7)
    out[fin] = np.rint(x[fin] / ulp) * ulp      # exact: ulp is a power of two
    out[np.abs(out) > 3.3961775e38] = np.inf * np.sign(out[np.abs(out) > 3.3961775e38])
    return out


def rope_frequencies(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, slow=1.0, fast=32.0):
    """Angle per position of each of the rot / 2 columns."""
    th = []
    for c in range(rot // 2):
        b = base * factor ** (rot / (rot - 2.0)) if scaling == "ntk" else base
        t = b ** (-2.0 * c / rot)
        if scaling == "linear":
            t /= factor
        if scaling == "by_parts":
            turns = orig_len * t / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            t = keep * t + (1 - keep) * t / factor
        th.append(t)
    return np.array(th)


def rope_tables(rows, rot, first=0, amplitude=1.0, **freq):
    ang = (first + np.arange(rows, dtype=np.float64))[:, None] * rope_frequencies(rot, **freq)[None]
    return amplitude * np.cos(ang), amplitude * np.sin(ang)


def rotate(x, cos, sin, interleaved=False, inverse=False):
    """x [N, H, d] turned by the angles of rows cos, sin [N, rot / 2]."""
    half = cos.shape[1]
    y = np.array(x, dtype=np.float64)
    for c in range(half):
        a, b = (2 * c, 2 * c + 1) if interleaved else (c, c + half)
        s = -sin[:, c] if inverse else sin[:, c]
        y[:, :, a] = x[:, :, a] * cos[:, c, None] + x[:, :, b] * s[:, None]
        y[:, :, b] = x[:, :, b] * cos[:, c, None] - x[:, :, a] * s[:, None]
    return y


def rms_norm(x, gain, eps):
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return y if gain is None else y * gain


def quantise(x):
    """Numbers 0..15 and scales (s, z) of rows [..., d], groups of 64."""
    g = x.reshape(*x.shape[:-1], -1, 64)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)   # NaN stays
    with np.errstate(all="ignore"):
        s = bf16((hi - lo) / 15.0)
        s = np.where(s < 1e-36, 0.0, s)
        z = bf16(lo + 8.0 * s)
        # a span that fp32 cannot hold counts as one that is not finite
        bad = ~(np.isfinite(s) & np.isfinite(z)) | (hi - lo >= 2.0 ** 128 - 2.0 ** 103)
        s, z = np.where(bad, np.nan, s), np.where(bad, np.nan, z)
        n = np.clip(np.floor((g - z) / np.where(s > 0, s, 1.0) + 8.5), 0, 15)
    n = np.where(s > 0, n, 8)
    return n.astype(np.int64).reshape(x.shape), s[..., 0], z[..., 0]


def dequantise(n, s, z):
    g = n.reshape(*n.shape[:-1], -1, 64)
    return (s[..., None] * (g - 8.0) + z[..., None]).reshape(n.shape)


def nibble_places(d):
    """(key, value) nibble index of each channel: in a token's row of keys, and
    of the even token in a pair's row of values (the odd one: + 4)."""
    G = d // 64
    key, val = [], []
    for c in range(d):
        g, x = divmod(c, 64)
        key.append(((x // 16) * G + g) * 16 + x % 16)
        val.append((((x // 8) * G + g) * 2 + x % 8 // 4) * 8 + x % 4)
    return np.array(key), np.array(val)


def to_bits16(x):
    """The bf16 bit patterns of float64 values that bf16 holds."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def put_nibble(row, index, n):
    b = index // 2
    row[b] = (row[b] & 0xF0 | n) if index % 2 == 0 else (row[b] & 0x0F | n << 4)


def write_row(cache, page, slot, h, key, value):
    """Puts one token's quantised key and value (n, s, z each) into cache
    uint8 [n_pages, Hkv, page / 16, 18 d]."""
    d = cache.shape[3] // 18
    G = d // 64
    off, t = slot % page, slot % 16
    tile = cache[slot // page, h, off // 16]
    kp, vp = nibble_places(d)
    for c in range(d):
        put_nibble(tile, t * d + int(kp[c]), int(key[0][c]))
        put_nibble(tile, 16 * d + (t // 2) * 2 * d + (t % 2) * 4 + int(vp[c]), int(value[0][c]))
    sc = tile[16 * d:].view(np.uint16)
    for which, (_, s, z) in enumerate((key, value)):
        for g in range(G):
            sc[((which * 16 + t) * G + g) * 2] = to_bits16(s[g])
            sc[((which * 16 + t) * G + g) * 2 + 1] = to_bits16(z[g])


def read_row(cache, page, slot, h):
    """key, value [d] held at a slot, float64."""
    d = cache.shape[3] // 18
    G = d // 64
    off, t = slot % page, slot % 16
    tile = cache[slot // page, h, off // 16]
    nib = np.empty(2 * tile.size, dtype=np.int64)
    nib[0::2], nib[1::2] = tile & 15, tile >> 4
    kp, vp = nibble_places(d)
    with np.errstate(invalid="ignore"):   # a NaN stays one
        sc = (tile[16 * d:].view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    sc = sc.reshape(2, 16, G, 2)
    k = dequantise(nib[t * d + kp], sc[0, t, :, 0], sc[0, t, :, 1])
    v = dequantise(nib[16 * d + (t // 2) * 2 * d + (t % 2) * 4 + vp], sc[1, t, :, 0], sc[1, t, :, 1])
    return k, v


def append_rows(k, v, gk=None, eps=1e-6, cos=None, sin=None, interleaved=False, ve_rows=None, gate=None, ve_scale=0.5):
    """What the append holds for keys and values [N, Hkv, d]: cos, sin
    [N, rot / 2] of the tokens' positions (None: no rotary), ve_rows [N, Hkv,
    d] their embeddings and gate [N, Hkv] (None: 1). Returns the exact rows
    and the held ones, key and value."""
    k = np.asarray(k, dtype=np.float64)
    v = np.asarray(v, dtype=np.float64)
    if cos is not None:
        k = rotate(k, cos, sin, interleaved)
    k = rms_norm(k, gk, eps)
    if ve_rows is not None:
        v = v + ve_scale * (1.0 if gate is None else gate[..., None]) * ve_rows
    return k, v, dequantise(*quantise(k)), dequantise(*quantise(v))


def attend(q, keys, values, window=-1, gq=None, eps=1e-6, scale=None, cos=None, sin=None, interleaved=False):
    """o [Hq, d], lse [Hq] of one request: q [Hq, d], keys and values [len,
    Hkv, d] (NaN keys or values outside the window are not looked at); cos,
    sin [rot / 2] of position len - 1."""
    Hq, d = q.shape
    n = len(keys)
    if n == 0:
        return np.zeros((Hq, d)), np.full(Hq, -np.inf)
    q = np.asarray(q, dtype=np.float64)
    if cos is not None:
        q = rotate(q[None], cos[None], sin[None], interleaved)[0]
    q = rms_norm(q, gq, eps)
    lo = 0 if window < 0 else max(0, n - 1 - window)
    keys, values = keys[lo:], values[lo:]
    G = Hq // keys.shape[1]
    scale = 1.0 / math.sqrt(d) if not scale else scale
    o, lse = np.zeros((Hq, d)), np.zeros(Hq)
    for h in range(Hq):
        z = scale * keys[:, h // G] @ q[h]
        m = z.max()
        p = np.exp(z - m)
        lse[h] = m + np.log(p.sum())
        o[h] = p @ values[:, h // G] / p.sum()
    return o, lse


def plan(lens, new, table, free, head, page, n_pages, n_tokens):
    """One request after the other. Returns a dict like the library's."""
    B, max_pages = table.shape
    table = table.copy()
    out = {"slot": np.full(n_tokens, -1, np.int64), "pos": np.zeros(n_tokens, np.int32),
           "row": np.full(n_tokens, -1, np.int32), "cu": np.zeros(B + 1, np.int32), "lens": lens.copy()}
    tok, asked, given, refused = 0, 0, 0, 0
    for b in range(B):
        n, m = int(lens[b]), int(new[b])
        ok = n >= 0 and m >= 0 and n + m <= max_pages * page
        m = max(m, 0)
        held = -(-n // page) if ok else 0
        want = -(-(n + m) // page) - held if ok else 0
        fits = ok and (want == 0 or head + asked + want <= len(free)) and tok + m <= n_tokens
        refused += not fits
        if fits:
            for i in range(want):
                table[b, held + i] = free[head + asked + i]
            if want:
                given = asked + want
            out["lens"][b] = n + m
        for i in range(m):
            if tok + i >= n_tokens:
                break
            t = n + i if n >= 0 and n + i < max_pages * page else 0
            out["row"][tok + i], out["pos"][tok + i] = b, t
            if fits and 0 <= table[b, t // page] < n_pages:
                out["slot"][tok + i] = int(table[b, t // page]) * page + t % page
        asked += want
        tok += m
        out["cu"][b + 1] = min(tok, 2 ** 31 - 1)
    out["table"], out["free_head"], out["refused"] = table, head + given, refused
    return out

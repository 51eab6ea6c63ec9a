"""GPU parity of the rotary and decode entry points against the float64
oracle (oracle/decode.py), for both builds.

Bounds (a rounding is off by at most half a step, u = 2^-24 in fp32):
  tables   the angle's 32-bit fraction becomes an fp32 number of half turns
           (u relative, at most pi u absolute), sincospif is good to 2 ulp:
           (pi + 4) u = 4.3e-7 absolute, times the amplitude.
  rotation half a step of the output, and four fp32 roundings of numbers no
           larger than |a| + |b|.
  append   values on plain layers enter the quantiser exactly, so the held
           numbers are the oracle's. Elsewhere fp32 rounding (32 u of the
           row's largest entry covers the rotation, the norm's sum over 128
           channels in a tree, rsqrt and two products) may move an entry
           across a border that close, and the span across a rounding border
           of its bf16 step: the step and centre are checked to be roundings
           of the exact ones within 64 u, and the numbers are then checked
           against the library's own step and centre.
  attend   with |q|, |k| norms up to 1.3 sqrt(d) and 2 sqrt(d) a logit's
           products sum to at most 30 in absolute value; the query's two fp16
           terms (2^-22), the norm (2^-21) and fp32 accumulation (16 steps of
           2^-23) make a logit wrong by at most 30 * 2.6e-6 = 8e-5: 1e-4 for
           lse (its own exp and log included), and, with P as two bf16 terms
           (2^-17), 2 * 8e-5 + 2^-17 = 1.7e-4 of the largest value for o, plus
           half a step of its type.
"""

import math

import numpy as np
import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from oracle import decode as dec

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": U}
EPS = 1e-6


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.detach().cpu().double().numpy()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen(seed)).to(dtype)


# ---------------------------------------------------------------------------
# Tables
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rot,rows,first,kw", [
    (128, 300, 0, {}),
    (16, 1, 0, {}),
    (48, 7, 1000003, {}),
    (64, 33, 2 ** 31 - 40, {}),                                   # the last positions there are
    (128, 50, 500000, dict(base=500000.0)),
    (96, 129, 12345, dict(scaling="linear", factor=4.0)),
    (128, 129, 200000, dict(scaling="ntk", factor=8.0)),
    (64, 257, 65536, dict(scaling="by_parts", factor=16.0, orig_len=4096, amplitude=1.25)),
    (16, 40, 77, dict(scaling="by_parts", factor=2.5, orig_len=300.0, slow=2.0, fast=8.0)),
    (32, 12, 5, dict(base=1.0)),                                  # every column one radian per position
])
def test_tables(rot, rows, first, kw):
    cos, sin = swa.rope_tables(rows, rot, first=first, **kw)
    rc, rs = dec.rope_tables(rows, rot, first=first, **kw)
    # the oracle's own angle, a float64 product, is off by first * 2^-53
    tol = (4.3e-7 + (first + rows) * 2.0 ** -52) * kw.get("amplitude", 1.0)
    assert cos.shape == (rows, rot // 2) and cos.dtype == torch.float32
    assert np.abs(f64(cos) - rc).max() <= tol
    assert np.abs(f64(sin) - rs).max() <= tol


def test_tables_serve_the_fused_rotation():
    # the attention with tables of swa_rope_tables, and rope_apply before the
    # attention without tables, are the same computation
    B, T, Hq, Hkv, d = 2, 150, 4, 2, 64
    q, k, v = (randn(i, B, T, h, d).to(dev()) for i, h in ((1, Hq), (2, Hkv), (3, Hkv)))
    rope = swa.rope_tables(T, d)
    o, lse, ws = swa.attention_forward(q, k, v, window=40, rope=rope)
    qr, kr = swa.rope_apply(q, k, rope)
    o2, lse2, ws2 = swa.attention_forward(qr, kr, v, window=40)
    assert (o - o2).abs().max().item() <= 1e-5 and (lse - lse2).abs().max().item() <= 1e-5
    dO = randn(4, B, T, Hq, d).to(dev())
    g = swa.attention_backward(q, k, v, None, None, o, lse, dO, window=40, rope=rope, workspace=ws, reuse_prologue=True)
    h = swa.attention_backward(qr, kr, v, None, None, o2, lse2, dO, window=40, workspace=ws2, reuse_prologue=True)
    dq, dk = swa.rope_apply(h["dq"], h["dk"], rope, inverse=True)
    for a, b in ((g["dq"], dq), (g["dk"], dk), (g["dv"], h["dv"])):
        assert (a - b).norm().item() <= 1e-5 * a.norm().item()


# ---------------------------------------------------------------------------
# Rotation
# ---------------------------------------------------------------------------

ROPES = [  # B, T, Hq, Hkv, d, rot, interleaved, given positions
    (2, 37, 4, 2, 128, 128, False, False),
    (1, 1, 1, 1, 64, 16, False, False),
    (3, 5, 6, 3, 128, 48, False, True),
    (1, 130, 16, 4, 128, 64, True, False),
    (2, 9, 2, 1, 64, 64, True, True),
    (1, 3, 5, 5, 64, 48, True, False),
    (1, 2000, 3, 1, 128, 112, False, True),
    (1, 70001, 1, 1, 64, 32, True, True),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,Hq,Hkv,d,rot,inter,given", ROPES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rotation(kind, B, T, Hq, Hkv, d, rot, inter, given, inverse):
    q, k = randn(1, B, T, Hq, d, dtype=DT[kind]), randn(2, B, T, Hkv, d, dtype=DT[kind])
    rows = T + 3
    cos, sin = (torch.tensor(x, dtype=torch.float32) for x in dec.rope_tables(rows, rot))
    pos = torch.randint(0, rows, (B, T), generator=gen(3), dtype=torch.int32) if given else None
    at = pos.numpy().ravel() if given else np.tile(np.arange(T), B)
    qd, kd, tabs = q.to(dev()), k.to(dev()), (cos.to(dev()), sin.to(dev()))
    pd = None if pos is None else pos.to(dev())
    qo, ko = swa.rope_apply(qd, kd, tabs, pos=pd, interleaved=inter, inverse=inverse)
    for x, y in ((q, qo), (k, ko)):
        a = f64(x).reshape(B * T, -1, d)
        c, s = f64(cos)[at], f64(sin)[at]
        ref = dec.rotate(a, c, s, inter, inverse)
        mag = np.abs(a) + np.abs(dec.rotate(a, 0 * c, 1 + 0 * s, inter))     # |a| + |b|
        tol = HALF[kind] * np.abs(ref) + 4 * U * mag
        err = np.abs(f64(y).reshape(ref.shape) - ref)
        assert np.all(err <= tol), float((err - tol).max())
        assert torch.equal(y.cpu().reshape(B * T, -1, d)[..., rot:], x.reshape(B * T, -1, d)[..., rot:])
    # in place, and one tensor alone, are the same bits
    q2, k2 = qd.clone(), kd.clone()
    swa.rope_apply(q2, k2, tabs, pos=pd, interleaved=inter, inverse=inverse, out=(q2, k2))
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    only = swa.rope_apply(None, kd, tabs, pos=pd, interleaved=inter, inverse=inverse)
    assert only[0] is None and torch.equal(only[1], ko)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_backward_is_the_formulas_and_the_differences(inter):
    # L = <g, R x>: dL/dx = R^T g, and (L(x + h e) - L(x - h e)) / 2h along random e
    B, T, H, d, rot = 1, 6, 2, 64, 48
    x, g, e = (randn(i, B, T, H, d).to(dev()) for i in (1, 2, 3))
    tabs = swa.rope_tables(T, rot)
    dx, _ = swa.rope_apply(g, None, tabs, interleaved=inter, inverse=True)
    h = 2.0 ** -3      # L is linear: any step serves
    up, _ = swa.rope_apply(x + h * e, None, tabs, interleaved=inter)
    dn, _ = swa.rope_apply(x - h * e, None, tabs, interleaved=inter)
    diff = float(((up.double() - dn.double()) * g.double()).sum()) / (2 * h)
    want = float((dx.double() * e.double()).sum())
    # 768 products of size ~1, each off by a few u / h
    assert abs(diff - want) <= 768 * 16 * 8 * U
    leaf = x.clone().requires_grad_(True)
    cos, sin = (t[None, :, None] for t in tabs)
    a, b = (leaf[..., 0:rot:2], leaf[..., 1:rot:2]) if inter else (leaf[..., :rot // 2], leaf[..., rot // 2:rot])
    ga, gb = (g[..., 0:rot:2], g[..., 1:rot:2]) if inter else (g[..., :rot // 2], g[..., rot // 2:rot])
    loss = ((a * cos + b * sin) * ga + (b * cos - a * sin) * gb).sum() + (leaf[..., rot:] * g[..., rot:]).sum()
    loss.backward()
    assert (leaf.grad - dx).abs().max().item() <= 16 * U * 8


def test_positions_outside_the_tables_are_left_and_reported():
    q = randn(1, 1, 5, 2, 64, dtype=torch.bfloat16).to(dev())
    tabs = swa.rope_tables(10, 64)
    pos = torch.tensor([[0, 10, -1, 9, 2 ** 31 - 1]], dtype=torch.int32, device=dev())
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    out = torch.full_like(q, 7.0)
    swa.rope_apply(q, None, tabs, pos=pos, out=(out, None), workspace=ws)
    assert swa.swa_attn_check_status(ws) == swa.SWA_ERR_DEVICE_CHECK
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK
    assert torch.all(out[0, [1, 2, 4]] == 7.0) and not torch.any(out[0, [0, 3]] == 7.0)
    swa.rope_apply(q, None, tabs, pos=pos.clamp(0, 9), workspace=ws)
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK
    with pytest.raises(swa.SwaError):
        swa.rope_apply(q, None, swa.rope_tables(4, 64))      # five positions counted from 0


# ---------------------------------------------------------------------------
# Append and read
# ---------------------------------------------------------------------------

def random_cache(seed, n_pages, Hkv, page, d):
    return torch.randint(0, 256, (n_pages, Hkv, page // 16, 18 * d), generator=gen(seed), dtype=torch.uint8)


def scales_of(cache, page, slot):
    """(s, z) [2 (key, value), Hkv, G] of a slot of a CPU cache, float64."""
    d = cache.shape[3] // 18
    tile = cache[slot // page, :, slot % page // 16, 16 * d:].contiguous().view(torch.bfloat16).double().numpy()
    sc = tile.reshape(cache.shape[1], 2, 16, d // 64, 2)[:, :, slot % 16]
    return sc.transpose(1, 0, 2, 3)


def numbers_of(cache, page, slot):
    d = cache.shape[3] // 18
    kp, vp = dec.nibble_places(d)
    t = slot % 16
    tile = cache[slot // page, :, slot % page // 16].numpy()
    nib = np.empty((tile.shape[0], 2 * tile.shape[1]), np.int64)
    nib[:, 0::2], nib[:, 1::2] = tile & 15, tile >> 4
    return nib[:, t * d + kp], nib[:, 16 * d + (t // 2) * 2 * d + (t % 2) * 4 + vp]


def check_held(x, n, s, z, exact_input, mag):
    """x [H, d] exact rows; n [H, d], s, z [H, G] as the library holds them."""
    H, d = x.shape
    g = x.reshape(H, -1, 64)
    m = np.broadcast_to(np.asarray(mag).reshape(H, 1, 1), (H, d // 64, 1))[..., 0]
    lo, hi = g.min(-1), g.max(-1)
    slack = 0.0 if exact_input else 64 * U * m
    raw = (hi - lo) / 15.0
    # fp32 rounds before bf16 does: 4 u more
    step = lambda v: 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 1e-30))) - 7)   # noqa: E731
    assert np.all(np.abs(s - raw) <= step(raw) / 2 + slack + 4 * U * np.abs(raw))
    rz = lo + 8 * s
    assert np.all(np.abs(z - rz) <= step(rz) / 2 + slack + 4 * U * (np.abs(rz) + np.abs(lo)))
    ng = n.reshape(g.shape).astype(np.float64)
    with np.errstate(all="ignore"):
        t = (g - z[..., None]) / s[..., None] + 8.5
        d_ = (0.0 if exact_input else 1.0) * (32 * U * (m[..., None] + np.abs(z[..., None])) / s[..., None])
    live = (s > 0)[..., None] & np.ones_like(g, dtype=bool)
    low = np.where(t - 1 - d_ <= 15, np.clip(np.floor(t - d_), 0, 15), 15)
    high = np.clip(np.floor(t + d_), 0, 15)
    assert np.all((ng >= low)[live]) and np.all((ng <= high)[live])
    assert np.all(ng[~live] == 8)


APPENDS = [  # B, T, Hkv, d, page, rot (0: none), interleaved, given pos, ve, gate
    (2, 21, 3, 128, 32, 128, False, True, False, None),
    (1, 1, 1, 64, 16, 0, False, False, False, None),
    (3, 17, 2, 64, 48, 64, True, True, True, "given"),
    (1, 40, 2, 128, 64, 48, False, False, True, None),
    (2, 9, 4, 128, 16, 32, True, True, True, "learned"),
    (5, 1, 6, 128, 128, 128, False, True, True, "learned"),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,Hkv,d,page,rot,inter,given,ve,gate", APPENDS)
def test_append_and_read(kind, B, T, Hkv, d, page, rot, inter, given, ve, gate):
    n_pages = B * T // page + 4
    before = random_cache(9, n_pages, Hkv, page, d)
    cache = before.to(dev())
    k, v = randn(1, B, T, Hkv, d, dtype=DT[kind]), randn(2, B, T, Hkv, d, dtype=DT[kind]) * 3
    if B > 1:
        k[1, 0] *= 1e-6
        v[1, 0] = 0.25       # constant groups
        v[0, 0] *= 1e20
    gk = 1 + 0.1 * randn(3, d)
    slots = torch.randperm(n_pages * page, generator=gen(4))[:B * T].view(B, T)
    if B * T > 3:
        slots[-1, -1] = -1
    rows = T + 9
    tabs = None if not rot else tuple(torch.tensor(x, dtype=torch.float32) for x in dec.rope_tables(rows, rot))
    pos = torch.randint(0, rows, (B, T), generator=gen(5), dtype=torch.int32) if given else None
    at = pos.numpy().ravel() if given else np.tile(np.arange(T), B)
    vocab, kw, g64, e64 = 13, {}, None, None
    if ve:
        tab = randn(6, vocab, Hkv * d, dtype=DT[kind])
        tok = torch.randint(0, vocab, (B, T), generator=gen(7), dtype=torch.int32)
        e64 = f64(tab)[tok.numpy().ravel()].reshape(B * T, Hkv, d)
        kw = dict(ve=tab.to(dev()), tok=tok.to(dev()), ve_scale=0.5)
        if gate == "given":
            gt = 2 * torch.sigmoid(randn(8, B, T, Hkv))
            kw["ve_gate"], g64 = gt.to(dev()), f64(gt).reshape(B * T, Hkv)
        if gate == "learned":
            gx, gw = randn(10, B, T, 40, dtype=DT[kind]), 0.25 * randn(11, Hkv, 32)
            kw["gate_x"], kw["gate_w"] = gx.to(dev()), gw.to(dev())
            g64 = 2 / (1 + np.exp(-(f64(gx)[..., :32].reshape(B * T, 32) @ f64(gw).T)))
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    dt = None if tabs is None else tuple(t.to(dev()) for t in tabs)
    swa.kv4_append(cache, k.to(dev()), v.to(dev()), slots.to(dev()), pos=None if pos is None else pos.to(dev()), rope=dt,
                   interleaved=inter, gk=gk.to(dev()), workspace=ws, **kw)
    kr, vr = swa.kv4_read(cache, slots.to(dev()), dtype=DT[kind], workspace=ws)
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK
    after = cache.cpu()
    rope64 = {} if tabs is None else dict(cos=f64(tabs[0])[at], sin=f64(tabs[1])[at])
    kx, vx, _, _ = dec.append_rows(f64(k).reshape(-1, Hkv, d), f64(v).reshape(-1, Hkv, d), f64(gk), EPS, interleaved=inter,
                                   ve_rows=e64, gate=g64, **rope64)
    kr, vr = f64(kr).reshape(-1, Hkv, d), f64(vr).reshape(-1, Hkv, d)
    touched = before.clone()
    for i, slot in enumerate(slots.flatten().tolist()):
        if slot < 0:
            assert np.all(kr[i] == 0) and np.all(vr[i] == 0)
            continue
        sc = scales_of(after, page, slot)
        nk, nv = numbers_of(after, page, slot)
        check_held(kx[i], nk, sc[0, :, :, 0], sc[0, :, :, 1], False, np.abs(kx[i]).max(-1))
        # with an embedding the value is a sum of two terms, and the gate is fp32
        mag = np.abs(vx[i]).max(-1) + (np.abs(e64[i]).max(-1) if ve else 0)
        check_held(vx[i], nv, sc[1, :, :, 0], sc[1, :, :, 1], kind == "bf16" and not ve, mag)
        for n, s, got in ((nk, sc[0], kr[i]), (nv, sc[1], vr[i])):
            want = dec.dequantise(n, s[..., 0], s[..., 1])
            assert np.all(np.abs(got - want) <= HALF[kind] * np.abs(want) + U * (15 * s[..., 0].repeat(64, -1) + np.abs(want)))
        tile = touched.numpy()
        for h in range(Hkv):
            dec.write_row(tile, page, slot, h, (nk[h], sc[0, h, :, 0], sc[0, h, :, 1]), (nv[h], sc[1, h, :, 0], sc[1, h, :, 1]))
    assert torch.equal(touched, after), "a byte of another slot changed"


def test_append_keeps_infinities_and_nans_apart():
    d, page = 128, 16
    cache = random_cache(1, 2, 1, page, d).to(dev())
    k, v = randn(1, 1, 4, 1, d, dtype=torch.bfloat16), randn(2, 1, 4, 1, d, dtype=torch.bfloat16)
    v[0, 1, 0, 5] = math.inf
    v[0, 2, 0, 70] = math.nan
    v[0, 3, 0, 64], v[0, 3, 0, 65] = 3e38, -3e38        # the span overflows
    k[0, 2, 0, 0] = math.nan                             # the norm spreads it over the row
    slot = torch.arange(4, device=dev()).view(1, 4)
    swa.kv4_append(cache, k.to(dev()), v.to(dev()), slot)
    kr, vr = (x[0, :, 0].float().cpu() for x in swa.kv4_read(cache, slot))
    nan = torch.isnan(vr)
    want = torch.zeros(4, d, dtype=torch.bool)
    want[1, :64] = want[2, 64:] = want[3, 64:] = True
    assert torch.equal(nan, want)
    assert torch.isnan(kr[2]).all() and torch.isfinite(kr[[0, 1, 3]]).all()


def test_append_refuses_on_the_device():
    d, page, n_pages = 64, 16, 3
    before = random_cache(1, n_pages, 2, page, d)
    k = randn(1, 1, 6, 2, d, dtype=torch.bfloat16).to(dev())
    tabs = swa.rope_tables(4, d)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    for slots, pos, tok, want in (
            ([0, 48, 2, -1, 4, 5], [0] * 6, None, [0, 2, 4, 5]), ([0, -2, 2 ** 62, 3, 4, -2 ** 63], [0] * 6, None, [0, 3, 4]),
            ([0, 1, 2, 3, 4, -1], [0, 4, -1, 3, 2 ** 31 - 1, 99], None, [0, 3]),
            ([0, 1, 2, 3, 4, 5], [0] * 6, [0, 5, -1, 1, 2, 2 ** 31 - 1], [0, 1, 2, 3, 4, 5])):
        cache = before.to(dev())
        kw = {}
        if tok is not None:
            kw = dict(ve=randn(4, 5, 2 * d, dtype=torch.bfloat16).to(dev()), tok=torch.tensor([tok], dtype=torch.int32, device=dev()))
        swa.kv4_append(cache, k, k, torch.tensor([slots], device=dev()), pos=torch.tensor([pos], dtype=torch.int32, device=dev()),
                       rope=tabs, workspace=ws, **kw)
        assert swa.swa_attn_check_status(ws) == swa.SWA_ERR_DEVICE_CHECK
        changed = [i for i, s in enumerate(slots) if 0 <= s < n_pages * page
                   and not np.array_equal(scales_of(cache.cpu(), page, s), scales_of(before, page, s))]
        assert changed == want
    cache = before.to(dev())
    swa.kv4_append(cache, k, k, torch.full((1, 6), -1, device=dev()), workspace=ws)
    assert torch.equal(cache.cpu(), before) and swa.swa_attn_check_status(ws) == swa.SWA_OK
    kr, vr = swa.kv4_read(cache, torch.tensor([[48, -1, -5]], device=dev()), workspace=ws)
    assert swa.swa_attn_check_status(ws) == swa.SWA_ERR_DEVICE_CHECK and not kr.any() and not vr.any()


# ---------------------------------------------------------------------------
# Plan
# ---------------------------------------------------------------------------

PLANS = [  # B, page, max_pages, longest, new (None: one each), pages missing, room for tokens behind
    (1, 16, 4, 30, None, 0, 0),
    (7, 16, 9, 100, 30, 0, 5),
    (64, 64, 20, 1000, None, 0, 0),
    (300, 48, 30, 1200, 200, 40, 3),
    (1025, 32, 12, 200, 9, 0, 1),
    (8192, 16, 6, 60, 2, 500, 7),
    (5, 128, 600, 70000, 6000, 10, 2),
]


@pytest.mark.parametrize("B,page,max_pages,longest,new,missing,extra", PLANS)
def test_plan(B, page, max_pages, longest, new, missing, extra):
    r = np.random.default_rng(B)
    cap = page * max_pages
    fresh = np.ones(B, np.int32) if new is None else np.where(r.random(B) < 0.2, 0, r.integers(0, new + 1, B)).astype(np.int32)
    lens = np.where(r.random(B) < 0.2, 0, r.integers(0, longest, B)).astype(np.int32)
    lens = np.minimum(lens, cap - fresh).astype(np.int32)
    held = -(-lens // page)
    n_pages = int(held.sum()) + B * max_pages + 8
    ids = r.permutation(n_pages).astype(np.int32)
    table = np.full((B, max_pages), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    want = int((-(-(lens.astype(np.int64) + fresh) // page) - held).sum())
    free, head = ids[at - min(at, 3):at + max(want - missing, 0)], min(at, 3)
    n_tokens = int(fresh.sum()) + extra
    ref = dec.plan(lens, fresh, table, free, head, page, n_pages, n_tokens)
    t = torch.tensor(table, device=dev())
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    out = swa.kv4_plan(torch.tensor(lens, device=dev()), None if new is None else torch.tensor(fresh, device=dev()), t,
                       torch.tensor(free, device=dev()), torch.tensor([head], dtype=torch.int32, device=dev()), page=page,
                       n_pages=n_pages, n_tokens=n_tokens, workspace=ws)
    assert (ref["refused"] > 0) == (missing > 0)
    assert swa.swa_attn_check_status(ws) == (swa.SWA_ERR_DEVICE_CHECK if missing else swa.SWA_OK)
    np.testing.assert_array_equal(t.cpu().numpy(), ref["table"])
    for x in ("slot", "pos", "row", "cu", "lens"):
        np.testing.assert_array_equal(out[x].cpu().numpy(), ref[x], err_msg=x)
    assert out["free_head"].item() == ref["free_head"]


def test_plan_refuses_on_the_device():
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev())   # noqa: E731
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())

    def run(lens, new, table, free, head, n_tokens, max_pages=4, n_pages=10):
        tab = np.array(table, np.int32).reshape(len(lens), max_pages)
        ref = dec.plan(np.array(lens, np.int32), np.array(new, np.int32), tab, np.array(free, np.int32), head, 16, n_pages, n_tokens)
        t = torch.tensor(tab, device=dev())
        out = swa.kv4_plan(i32(*lens), i32(*new), t, i32(*free), i32(head), page=16, n_pages=n_pages, n_tokens=n_tokens,
                           workspace=ws)
        np.testing.assert_array_equal(t.cpu().numpy(), ref["table"])
        for x in ("slot", "pos", "row", "cu", "lens"):
            np.testing.assert_array_equal(out[x].cpu().numpy(), ref[x], err_msg=x)
        assert out["free_head"].item() == ref["free_head"]
        return swa.swa_attn_check_status(ws)

    bad = swa.SWA_ERR_DEVICE_CHECK
    row = [[0, 1, 2, 3], [4, 5, 6, 7]]
    assert run([60, 3], [5, 1], row, [8, 9], 0, 8) == bad                 # past its table row
    assert run([-1, 3], [1, 1], row, [8, 9], 0, 8) == bad
    assert run([3, 3], [-4, 1], row, [8, 9], 0, 8) == bad
    assert run([2 ** 31 - 1, 3], [2 ** 31 - 1, 1], row, [8, 9], 0, 8) == bad
    assert run([3, 3], [4, 5], row, [8, 9], 0, 8) == bad                  # nine tokens, room for eight
    assert run([20, 3], [1, 1], [[0, 99, -1, -1], [4, -1, -1, -1]], [8, 9], 0, 2) == bad   # a page that is not there
    assert run([16, 3], [1, 1], row, [77, 9], 0, 2) == bad                # a free page that is not there
    assert run([16, 3], [1, 1], row, [8, 9], 2, 2) == bad                 # none left
    assert run([16, 3], [1, 1], row, [8, 9], 1, 2) == swa.SWA_OK
    assert run([0, 0], [0, 0], row, [8], 0, 0) == swa.SWA_OK
    out = swa.kv4_plan(i32(), None, torch.zeros(0, 4, dtype=torch.int32, device=dev()), i32(1), i32(0), page=16, n_pages=4,
                       n_tokens=3)
    assert out["slot"].tolist() == [-1] * 3 and out["cu"].tolist() == [0] and out["free_head"].tolist() == [0]


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def build_cache(lens, Hkv, d, page, seed=1, spare=2):
    """A CPU cache with random rows in [0, len) of each request, NaN scales
    and arbitrary numbers everywhere else; its table; keys, values per request."""
    held = [-(-n // page) for n in lens]
    n_pages = sum(held) + spare
    g = torch.Generator().manual_seed(seed)
    cache = torch.randint(0, 256, (n_pages, Hkv, page // 16, 18 * d), generator=g, dtype=torch.uint8)
    G = d // 64
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(n_pages, Hkv, page // 16, 2, 16, G, 2)
    good = torch.stack([0.15 + 0.1 * torch.rand(sc.shape[:-1], generator=g), 0.2 * torch.randn(sc.shape[:-1], generator=g)], -1)
    ids = torch.randperm(n_pages, generator=g)
    width = max(held + [1]) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at, rows = 0, []
    sc[:] = math.nan
    for b, n in enumerate(lens):
        table[b, :held[b]] = ids[at:at + held[b]].int()
        at += held[b]
        for j in range(n):
            pg, off = int(table[b, j // page]), j % page
            sc[pg, :, off // 16, :, off % 16] = good[pg, :, off // 16, :, off % 16].bfloat16()
        slots = [int(table[b, j // page]) * page + j % page for j in range(n)]
        kv = [numbers_of(cache, page, s) + (scales_of(cache, page, s),) for s in slots]
        keys = np.array([dec.dequantise(nk, s[0, :, :, 0], s[0, :, :, 1]) for nk, _, s in kv]).reshape(n, Hkv, d)
        vals = np.array([dec.dequantise(nv, s[1, :, :, 0], s[1, :, :, 1]) for _, nv, s in kv]).reshape(n, Hkv, d)
        rows.append((keys, vals))
    return cache, table, rows


def check_attention(kind, lens, Hq, Hkv, d, page, window=-1, rot=0, inter=False, gain=True, scale=0.0, seed=1, factor=1.0,
                    workspace=None, stream=None):
    cache, table, rows = build_cache(lens, Hkv, d, page, seed)
    q = randn(seed + 1, len(lens), Hq, d, dtype=DT[kind]) * factor
    gq = 1 + 0.1 * randn(seed + 2, d) if gain else None
    n_rows = max(lens + [1])
    tabs = None if not rot else tuple(torch.tensor(x, dtype=torch.float32) for x in dec.rope_tables(n_rows, rot))
    cd = cache.to(dev())
    ws = workspace if workspace is not None else swa.new_kv4_workspace(cd, len(lens), Hq, max_pages=table.shape[1], window=window,
                                                                       kind=kind)
    o, lse = swa.kv4_attention(cd, q.to(dev()), table.to(dev()), torch.tensor(lens, dtype=torch.int32, device=dev()),
                               rope=None if tabs is None else tuple(t.to(dev()) for t in tabs), interleaved=inter,
                               gq=None if gq is None else gq.to(dev()), window=window, softmax_scale=scale, workspace=ws)
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    assert torch.equal(cd.cpu(), cache)
    o, lse = f64(o), f64(lse)
    for b, n in enumerate(lens):
        kw = {} if tabs is None or n == 0 else dict(cos=f64(tabs[0])[n - 1], sin=f64(tabs[1])[n - 1], interleaved=inter)
        ro, rl = dec.attend(f64(q)[b], *rows[b], window=window, gq=None if gq is None else f64(gq), scale=scale, **kw)
        if n == 0:
            assert np.all(o[b] == 0) and np.all(lse[b] == -np.inf)
            continue
        assert np.all(np.abs(lse[b] - rl) <= 1e-4), float(np.abs(lse[b] - rl).max())
        top = np.abs(rows[b][1]).max()
        tol = HALF[kind] * np.abs(ro) + 1.7e-4 * top
        assert np.all(np.abs(o[b] - ro) <= tol), float((np.abs(o[b] - ro) - tol).max())


LENS = [1, 0, 2, 15, 16, 17, 31, 32, 33, 47, 64, 65, 100, 127, 129, 200]
ATTENDS = [  # lens, Hq, Hkv, d, page, window, rot, interleaved
    (LENS, 4, 2, 128, 16, -1, 128, False),
    (LENS, 2, 1, 64, 48, -1, 64, False),
    (LENS, 6, 3, 128, 64, 40, 128, False),
    (LENS, 3, 3, 64, 32, 0, 32, True),
    (LENS, 3, 1, 128, 128, 15, 0, False),
    (LENS, 5, 1, 64, 16, 16, 16, False),
    (LENS, 8, 1, 128, 32, 17, 96, False),
    (LENS, 9, 1, 64, 32, -1, 48, True),
    (LENS, 17, 1, 128, 16, 1, 64, True),
    ([1500, 3, 777, 0], 4, 1, 128, 64, -1, 128, False),
    ([2500], 2, 2, 64, 16, -1, 64, False),
    ([2048, 2049, 1], 2, 2, 128, 256, 1000, 128, False),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,rot,inter", ATTENDS)
def test_attention(kind, lens, Hq, Hkv, d, page, window, rot, inter):
    check_attention(kind, lens, Hq, Hkv, d, page, window, rot, inter)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_attention_without_gain_and_with_a_scale(kind):
    check_attention(kind, [70, 5], 4, 2, 128, 32, gain=False, scale=0.05)
    check_attention(kind, [70, 5], 2, 2, 64, 16, gain=False, rot=64)
    # the norm takes the query's size out (eps aside): very large and small ones
    check_attention(kind, [40], 2, 2, 64, 16, factor=1e15)
    check_attention(kind, [40], 2, 2, 64, 16, factor=1e-2)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_attention_of_values_of_very_different_size(kind):
    # the steps of the values span 60 powers of two, one large value among
    # tokens that hardly count: nothing overflows, underflows or drowns
    d, page, n = 128, 32, 90
    cache, table, _ = build_cache([n], 1, d, page)
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(-1, 1, page // 16, 2, 16, 2, 2)
    exps = torch.randint(-30, 30, (n,), generator=gen(3))
    for j in range(n):
        pg, off = int(table[0, j // page]), j % page
        sc[pg, 0, off // 16, 1, off % 16, :, 0] = 2.0 ** float(exps[j])
    rows = [numbers_of(cache, page, int(table[0, j // page]) * page + j % page)
            + (scales_of(cache, page, int(table[0, j // page]) * page + j % page),) for j in range(n)]
    keys = np.array([dec.dequantise(a, s[0, :, :, 0], s[0, :, :, 1]) for a, _, s in rows])
    vals = np.array([dec.dequantise(b, s[1, :, :, 0], s[1, :, :, 1]) for _, b, s in rows])
    q = randn(5, 1, 2, d, dtype=DT[kind])
    o, lse = swa.kv4_attention(cache.to(dev()), q.to(dev()), table.to(dev()), torch.tensor([n], dtype=torch.int32, device=dev()))
    ro, rl = dec.attend(f64(q)[0], keys, vals)
    qn = dec.rms_norm(f64(q)[0], None, EPS)
    z = qn @ keys[:, 0].T / math.sqrt(d)
    p = np.exp(z - z.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    weight = p @ np.abs(vals[:, 0])
    assert np.abs(f64(lse)[0] - rl).max() <= 1e-4
    assert np.all(np.abs(f64(o)[0] - ro) <= HALF[kind] * np.abs(ro) + 1.7e-4 * weight)


def test_attention_reports_what_it_leaves_out():
    lens = [40, 40, 40, 40]
    cache, table, rows = build_cache(lens, 1, 64, 16)
    cd = cache.to(dev())
    ws = swa.new_kv4_workspace(cd, 4, 2, max_pages=table.shape[1])
    q = randn(2, 4, 2, 64, dtype=torch.bfloat16)
    tabs = swa.rope_tables(40, 64)

    def run(t, n, rope=None):
        o, lse = swa.kv4_attention(cd, q.to(dev()), t.to(dev()), torch.tensor(n, dtype=torch.int32, device=dev()), rope=rope,
                                   workspace=ws)
        return f64(o), f64(lse), swa.swa_attn_check_status(ws)

    good = run(table, lens)
    assert good[2] == swa.SWA_OK
    bad = table.clone()
    bad[1, 1], bad[2, 0] = cache.shape[0], -3           # pages that are not there
    o, lse, st = run(bad, lens)
    assert st == swa.SWA_ERR_DEVICE_CHECK
    for b, keep in ((0, range(40)), (1, [*range(16), *range(32, 40)]), (2, range(16, 40))):
        ro, rl = dec.attend(f64(q)[b], rows[b][0][list(keep)], rows[b][1][list(keep)])
        assert np.abs(lse[b] - rl).max() <= 1e-4 and np.abs(o[b] - ro).max() <= 2.0 ** -8 * np.abs(ro).max() + 1.7e-4 * 4
    bad[3] = 2 ** 31 - 1                                 # none of its pages
    o, lse, st = run(bad, lens)
    assert st == swa.SWA_ERR_DEVICE_CHECK and np.all(o[3] == 0) and np.all(lse[3] == -np.inf)
    # a length below 0, one past the rotary tables, one past the table row
    o, lse, st = run(table, [-5, 40, 40, 40])
    assert st == swa.SWA_ERR_DEVICE_CHECK and np.all(o[0] == 0) and np.all(lse[0] == -np.inf)
    np.testing.assert_array_equal(o[1:], good[0][1:])
    o, lse, st = run(table, [41, 40, 40, 40], rope=tabs)
    assert st == swa.SWA_ERR_DEVICE_CHECK and np.all(o[0] == 0) and np.all(lse[0] == -np.inf)
    o, lse, st = run(table[:, :3].contiguous(), [2 ** 31 - 1, 40, 40, 40])
    assert st == swa.SWA_ERR_DEVICE_CHECK
    np.testing.assert_array_equal(o[1:], good[0][1:])


def test_a_nan_stays_in_its_request():
    lens = [40, 40]
    cache, table, _ = build_cache(lens, 2, 64, 16)
    sc = cache[..., 16 * 64:].view(torch.bfloat16).view(-1, 2, 1, 2, 16, 1, 2)
    sc[int(table[0, 1]), 1, 0, 0, 3] = math.nan          # one key of request 0, kv head 1
    q = randn(2, 2, 4, 64, dtype=torch.bfloat16).to(dev())
    args = (q, table.to(dev()), torch.tensor(lens, dtype=torch.int32, device=dev()))
    o, lse = swa.kv4_attention(cache.to(dev()), *args)
    nan = torch.isnan(o).all(-1).cpu()
    assert nan.tolist() == [[False, False, True, True], [False] * 4]
    assert torch.isfinite(o[1]).all() and torch.isfinite(o[0, :2]).all()
    o, lse = swa.kv4_attention(cache.to(dev()), *args, window=10)       # behind the window: not seen
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    o, lse = swa.kv4_attention(cache.to(dev()), torch.full_like(q, math.nan), *args[1:])
    assert torch.isnan(o).all()


def test_long_request_split_over_many_blocks_repeats_its_bits():
    # 8000 keys for one request: the parts are joined in a fixed order
    d, page, n = 128, 64, 8000
    n_pages = n // page + 2
    cache = random_cache(3, n_pages, 2, page, d)
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc[..., 0::2] = 0.2
    sc[..., 1::2] = (0.2 * randn(4, *sc[..., 1::2].shape)).bfloat16()
    cache = cache.to(dev())
    table = torch.randperm(n_pages, generator=gen(5))[None].int().to(dev())
    lens = torch.tensor([n], dtype=torch.int32, device=dev())
    q = randn(6, 1, 4, d, dtype=torch.bfloat16).to(dev())
    ws = swa.new_kv4_workspace(cache, 1, 4, max_pages=n_pages)
    runs = [swa.kv4_attention(cache, q, table, lens, workspace=ws) for _ in range(5)]
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    slot = (table[0].long()[:, None] * page + torch.arange(page, device=dev())).view(1, -1)[:, :n].contiguous()
    k, v = (x[0].double().cpu().numpy() for x in swa.kv4_read(cache, slot, dtype=torch.float32))
    ro, rl = dec.attend(f64(q)[0], k, v)
    o, lse = runs[0]
    assert np.abs(f64(lse)[0] - rl).max() <= 1e-4
    assert np.all(np.abs(f64(o)[0] - ro) <= 2.0 ** -8 * np.abs(ro) + 1.7e-4 * np.abs(v).max())
    for w in (0, 100, 5000):
        o, lse = swa.kv4_attention(cache, q, table, lens, window=w)
        ro, rl = dec.attend(f64(q)[0], k, v, window=w)
        assert np.abs(f64(lse)[0] - rl).max() <= 1e-4
        assert np.all(np.abs(f64(o)[0] - ro) <= 2.0 ** -8 * np.abs(ro) + 1.7e-4 * np.abs(v).max())


def test_one_workspace_serves_calls_of_other_shapes():
    # a few long requests (split, partial results), many short ones, long ones
    # again: nothing of one call is taken for another's
    shapes = [([3000, 2900], 4, 2, 128, 64), ([30] * 300, 4, 2, 128, 16), ([1800], 9, 1, 64, 32), ([2000, 5, 0, 700], 2, 2, 64, 16)]
    sizes = [swa.swa_kv4_workspace_size(swa.make_params(len(x), 1, hq, hkv, d), page, max(-(-n // page) for n in x) + 1)
             for x, hq, hkv, d, page in shapes]
    ws = torch.full((max(sizes),), 255, dtype=torch.uint8, device=dev())
    assert swa.swa_kv4_workspace_init(ws) == swa.SWA_OK
    for i in (0, 1, 2, 3, 1, 0, 3, 2):
        lens, Hq, Hkv, d, page = shapes[i]
        check_attention("bf16", lens, Hq, Hkv, d, page, workspace=ws, seed=10 + i)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_waits_that_run_out_are_reported_and_the_workspace_stays_usable(kind):
    # a limit of 1 ns, on requests whose 150 MB all come from memory: the
    # copies all land, only later than the limit allows
    d, page, n, Hkv, Hq, B = 128, 64, 8192, 2, 4, 64
    per = n // page
    cache = torch.randint(0, 256, (B * per, Hkv, page // 16, 18 * d), dtype=torch.uint8, device=dev())
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc[..., 0::2], sc[..., 1::2] = 0.2, 0.1
    table = torch.arange(B * per, dtype=torch.int32, device=dev()).view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev())
    q = randn(6, B, Hq, d, dtype=DT[kind]).to(dev())
    ws = swa.new_kv4_workspace(cache, B, Hq, max_pages=per, kind=kind)
    want = swa.kv4_attention(cache, q, table, lens, workspace=ws)
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    p, c = swa.make_params(B, 1, Hq, Hkv, d), swa.swa_kv4_cache(cache.data_ptr(), B * per, page)
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device=dev())
    short = swa.make_extras(wait_limit_ns=1)
    for _ in range(3):
        st = swa.swa_kv4_attn(p, short, c, None, q, None, table, per, lens, o, lse, ws)
        assert st == swa.SWA_OK
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_ERR_TIMEOUT
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK      # read and cleared
        got = swa.kv4_attention(cache, q, table, lens, workspace=ws)
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_cache_past_32_bits():
    # pages whose byte offsets, and slots, need more than 32 bits
    d, page, Hkv = 64, 512, 1
    per = Hkv * page // 16 * 18 * d
    n_pages = (1 << 32) // per + 40
    cache = torch.empty(n_pages, Hkv, page // 16, 18 * d, dtype=torch.uint8, device=dev())
    last = n_pages - 1
    cache[:2] = 255
    cache[-3:] = 255
    T = 30
    k, v = randn(1, 1, T, Hkv, d, dtype=torch.bfloat16).to(dev()), randn(2, 1, T, Hkv, d, dtype=torch.bfloat16).to(dev())
    slot = last * page + page - T + torch.arange(T, device=dev()).view(1, T)
    swa.kv4_append(cache, k, v, slot)
    assert torch.all(cache[:2] == 255)
    small = torch.full((1, Hkv, page // 16, 18 * d), 255, dtype=torch.uint8, device=dev())
    swa.kv4_append(small, k, v, slot - last * page)
    assert torch.equal(cache[last], small[0])
    a, b = swa.kv4_read(cache, slot), swa.kv4_read(small, slot - last * page)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    lens = torch.tensor([page], dtype=torch.int32, device=dev())
    q = randn(3, 1, 2, d, dtype=torch.bfloat16).to(dev())
    one = [swa.kv4_attention(c, q, torch.tensor([[p]], dtype=torch.int32, device=dev()), lens, window=T - 1)
           for c, p in ((cache, last), (small, 0))]
    assert torch.equal(one[0][0], one[1][0]) and torch.isfinite(one[0][0]).all()


# ---------------------------------------------------------------------------
# Together, as a serving loop uses them
# ---------------------------------------------------------------------------

def test_serving_steps():
    """Prompts of four requests, then single tokens, through plan, append and
    attention on one layer with value embeddings and a window: every step's
    output against the oracle on all rows as the cache holds them, and the
    held rows against the exact ones."""
    Hq, Hkv, d, page, window, vocab = 6, 3, 128, 32, 50, 19
    prompts, steps = [37, 1, 64, 90], 4
    B, total = len(prompts), sum(prompts)
    n_pages = 40
    cache = torch.full((n_pages, Hkv, page // 16, 18 * d), 255, dtype=torch.uint8, device=dev())
    free = torch.randperm(n_pages, generator=gen(1)).int().to(dev())
    head = torch.zeros(1, dtype=torch.int32, device=dev())
    table = torch.full((B, 6), -1, dtype=torch.int32, device=dev())
    lens = torch.zeros(B, dtype=torch.int32, device=dev())
    tabs = swa.rope_tables(128, d)
    gq, gk = (1 + 0.1 * randn(i, d) for i in (2, 3))
    tab = randn(4, vocab, Hkv * d, dtype=torch.bfloat16)
    ws = swa.new_kv4_workspace(cache, B, Hq, max_pages=6, window=window)
    seen = [[] for _ in range(B)]      # exact (k, v) rows of each request

    def step(new, seed):
        nonlocal lens, head
        n = sum(new)
        k, v = (randn(seed + i, n, 1, Hkv, d, dtype=torch.bfloat16) for i in (0, 1))
        tok = torch.randint(0, vocab, (n, 1), generator=gen(seed + 2), dtype=torch.int32)
        plan = swa.kv4_plan(lens, torch.tensor(new, dtype=torch.int32, device=dev()), table, free, head, page=page,
                            n_pages=n_pages, n_tokens=n, workspace=ws)
        lens, head = plan["lens"], plan["free_head"]
        swa.kv4_append(cache, k.to(dev()), v.to(dev()), plan["slot"].view(n, 1), pos=plan["pos"].view(n, 1), rope=tabs,
                       gk=gk.to(dev()), ve=tab.to(dev()), tok=tok.to(dev()), workspace=ws)
        pos = plan["pos"].cpu().numpy()
        kx, vx, _, _ = dec.append_rows(f64(k)[:, 0], f64(v)[:, 0], f64(gk), EPS, f64(tabs[0])[pos], f64(tabs[1])[pos],
                                       ve_rows=f64(tab)[tok.numpy().ravel()].reshape(n, Hkv, d))
        for i, b in enumerate(plan["row"].tolist()):
            assert pos[i] == len(seen[b])
            seen[b].append((kx[i], vx[i]))

    step(prompts, 10)
    for s in range(steps):
        step([1] * B, 20 + 10 * s)
        q = randn(100 + s, B, Hq, d, dtype=torch.bfloat16)
        o, lse = swa.kv4_attention(cache, q.to(dev()), table, lens, rope=tabs, gq=gq.to(dev()), window=window, workspace=ws)
        assert swa.swa_attn_check_status(ws) == swa.SWA_OK
        for b in range(B):
            n = prompts[b] + s + 1
            assert lens[b].item() == n == len(seen[b])
            at = torch.arange(n, device=dev())
            slot = (table[b].long()[at // page] * page + at % page).view(1, n)
            kh, vh = (f64(x)[0] for x in swa.kv4_read(cache, slot, dtype=torch.float32))
            for held, j in ((kh, 0), (vh, 1)):
                exact = np.array([r[j] for r in seen[b]])
                span = np.ptp(exact.reshape(n, Hkv, -1, 64), axis=-1).repeat(64, -1).reshape(n, Hkv, d)
                assert np.all(np.abs(held - exact) <= span / 30 * 1.1 + 2.0 ** -7 * (np.abs(exact) + span))
            ro, rl = dec.attend(f64(q)[b], kh, vh, window=window, gq=f64(gq), cos=f64(tabs[0])[n - 1], sin=f64(tabs[1])[n - 1])
            assert np.abs(f64(lse)[b] - rl).max() <= 1e-4
            assert np.all(np.abs(f64(o)[b] - ro) <= 2.0 ** -8 * np.abs(ro) + 1.7e-4 * np.abs(vh).max())
    assert total + steps * B == sum(len(x) for x in seen)


def test_a_step_captured_and_replayed():
    """Plan, append and attention of a padded batch in one CUDA graph, replayed
    with new inputs, equal eager calls on the same inputs."""
    B, Hq, Hkv, d, page, max_pages, n_pages = 6, 4, 2, 64, 16, 8, 60
    i32 = dict(dtype=torch.int32, device=dev())
    tabs = swa.rope_tables(128, d)

    def state(seed):
        lens = torch.randint(0, 100, (B,), generator=gen(seed)).int()
        lens[2] = 0
        new = torch.ones(B, dtype=torch.int32)
        new[4] = 0                                    # a request that waits: its token slot is padding at the end
        held = -(-lens // page)
        ids = torch.randperm(n_pages, generator=gen(seed + 1)).int()
        table, at = torch.full((B, max_pages), -1, dtype=torch.int32), 0
        for b in range(B):
            table[b, :held[b]] = ids[at:at + int(held[b])]
            at += int(held[b])
        cache = random_cache(seed + 2, n_pages, Hkv, page, d)
        sc = cache[..., 16 * d:].view(torch.bfloat16)
        sc[..., 0::2], sc[..., 1::2] = 0.2, 0.1
        return [x.to(dev()) for x in (lens, new, table, ids[at:at + 8].clone(), torch.zeros(1, dtype=torch.int32), cache,
                                      randn(seed + 3, B, Hq, d, dtype=torch.bfloat16), randn(seed + 4, B, 1, Hkv, d, dtype=torch.bfloat16),
                                      randn(seed + 5, B, 1, Hkv, d, dtype=torch.bfloat16))]

    def step(s, ws):
        lens, new, table, free, head, cache, q, k, v = s
        plan = swa.kv4_plan(lens, new, table, free, head, page=page, n_pages=n_pages, n_tokens=B, workspace=ws)
        swa.kv4_append(cache, k, v, plan["slot"].view(B, 1), pos=plan["pos"].view(B, 1), rope=tabs, workspace=ws)
        o, lse = swa.kv4_attention(cache, q, table, plan["lens"], rope=tabs, workspace=ws)
        return [plan["slot"], plan["pos"], plan["row"], plan["cu"], plan["lens"], plan["free_head"], table, cache, o, lse]

    live = state(1)
    ws = swa.new_kv4_workspace(live[5], B, Hq, max_pages=max_pages)
    step([x.clone() for x in live], ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(live, ws)
    for seed in (1, 50, 99):
        fresh = state(seed)
        for a, b in zip(live, fresh):
            a.copy_(b)
        graph.replay()
        got = [x.clone() for x in out]
        want = step(fresh, swa.new_kv4_workspace(fresh[5], B, Hq, max_pages=max_pages))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert swa.swa_attn_check_status(ws) == swa.SWA_OK
        assert got[0][-1].item() == -1                # padding behind the last token


def test_two_streams_at_once():
    lens = [300, 40, 5]
    cache, table, _ = build_cache(lens, 2, 128, 32)
    cd, td = cache.to(dev()), table.to(dev())
    ld = torch.tensor(lens, dtype=torch.int32, device=dev())
    qs = [randn(i, 3, 4, 128, dtype=torch.bfloat16).to(dev()) for i in range(2)]
    want = [swa.kv4_attention(cd, q, td, ld) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    wss = [swa.new_kv4_workspace(cd, 3, 4, max_pages=td.shape[1]) for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (s, q) in enumerate(zip(streams, qs)):
            got[i].append(swa.kv4_attention(cd, q, td, ld, workspace=wss[i] if i else None, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    # by a raw handle, and rope and append on a side stream
    o, _ = swa.kv4_attention(cd, qs[0], td, ld, stream=streams[0].cuda_stream)
    tabs = swa.rope_tables(16, 64, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(o, want[0][0])
    ref = swa.rope_tables(16, 64)
    assert torch.equal(tabs[0], ref[0]) and torch.equal(tabs[1], ref[1])


def test_several_query_tokens_of_a_request_are_rows():
    # the same table row with lengths one apart
    cache, table, rows = build_cache([80], 2, 64, 16)
    n = 5
    lens = torch.arange(80 - n + 1, 81, dtype=torch.int32, device=dev())
    q = randn(3, n, 4, 64, dtype=torch.bfloat16)
    o, lse = swa.kv4_attention(cache.to(dev()), q.to(dev()), table.repeat(n, 1).to(dev()), lens)
    for i in range(n):
        m = 80 - n + 1 + i
        ro, rl = dec.attend(f64(q)[i], rows[0][0][:m], rows[0][1][:m])
        assert np.abs(f64(lse)[i] - rl).max() <= 1e-4
        assert np.all(np.abs(f64(o)[i] - ro) <= 2.0 ** -8 * np.abs(ro) + 1.7e-4 * np.abs(rows[0][1]).max())


# ---------------------------------------------------------------------------
# The short way of the binding
# ---------------------------------------------------------------------------

def test_short_way_is_there_and_gives_the_same_bits(monkeypatch):
    assert swa._fast is not None, "_fast.so is not built: the decode calls run the long way"
    swa.load("bf16"), swa.load("fp32")      # loading a library ties it to the module
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 16
    lens = torch.tensor([20, 0, 33], dtype=torch.int32, device=dev())
    new = torch.tensor([2, 40, 1], dtype=torch.int32, device=dev())
    table0 = torch.arange(24, dtype=torch.int32, device=dev()).view(3, 8)
    free = torch.arange(40, 60, dtype=torch.int32, device=dev())
    head = torch.zeros(1, dtype=torch.int32, device=dev())
    gq, gk = (1 + 0.1 * randn(i, d).to(dev()) for i in (1, 2))
    tab, gate = randn(3, 11, Hkv * d).to(dev()), torch.rand(43, 1, Hkv, device=dev())
    tok = torch.randint(0, 11, (43, 1), dtype=torch.int32, device=dev())
    taken = []
    kinds = {"bf16": torch.bfloat16, "fp32": torch.float32}

    class Watch:      # notes which calls the short way took
        def __getattr__(self, name):
            f = getattr(fast, name)

            def call(*a):
                r = f(*a)
                taken.append((name, r is not None))
                return r
            return call

    fast = swa._fast

    def everything(dt):
        rope = swa.rope_tables(64, 32, base=5000.0, scaling="by_parts", factor=3.0, orig_len=40)
        table = table0.clone()
        plan = swa.kv4_plan(lens, new, table, free, head, page=page, n_pages=60, n_tokens=43)
        one = swa.kv4_plan(lens, None, table, free, head, page=page, n_pages=60, n_tokens=5)
        cache = torch.zeros(60, Hkv, 1, 18 * d, dtype=torch.uint8, device=dev())
        ws = swa.new_kv4_workspace(cache, B, Hq, max_pages=8, kind="fp32" if dt is torch.float32 else "bf16")
        k, v, q = (randn(i, *s, dtype=dt).to(dev()) for i, s in ((4, (43, 1, Hkv, d)), (5, (43, 1, Hkv, d)), (6, (B, Hq, d))))
        slot, pos = plan["slot"].view(43, 1), plan["pos"].view(43, 1)
        swa.kv4_append(cache, k, v, slot, pos=pos, rope=rope, interleaved=True, gk=gk, ve=tab.to(dt), tok=tok, ve_gate=gate,
                       ve_scale=0.25, eps=1e-3, workspace=ws)
        swa.kv4_append(cache, k[:1], v[:1], slot[:1])
        kr, vr = swa.kv4_read(cache, slot, dtype=dt)
        att = swa.kv4_attention(cache, q, table, plan["lens"], rope=rope, interleaved=True, gq=gq, window=30,
                                softmax_scale=0.1, eps=1e-3, workspace=ws)
        bare = swa.kv4_attention(cache, q, table, plan["lens"], workspace=ws)
        x = randn(7, B, 9, Hq, d, dtype=dt).to(dev())
        turned = swa.rope_apply(x, x[:, :, :Hkv].contiguous(), rope)
        back = swa.rope_apply(x, None, rope, pos=torch.full((B, 9), 5, dtype=torch.int32, device=dev()), interleaved=True, inverse=True)
        swa.rope_apply(None, x, rope, out=(None, x))
        return [*rope, *plan.values(), *one.values(), table, cache, kr, vr, *att, *bare, *turned, back[0], x]

    for dt in kinds.values():
        monkeypatch.setattr(swa, "_fast", None)
        want = everything(dt)
        monkeypatch.setattr(swa, "_fast", Watch())
        taken.clear()
        got = everything(dt)
        assert len(taken) == 11 and all(ok for _, ok in taken), taken
        for a, b in zip(got, want):
            assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)


def test_short_way_leaves_the_unusual_to_the_long_one():
    c = torch.zeros(4, 2, 1, 18 * 64, dtype=torch.uint8, device=dev())
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=dev())
    table, lens = torch.zeros(1, 4, dtype=torch.int32, device=dev()), torch.ones(1, dtype=torch.int32, device=dev())
    ws = swa.new_kv4_workspace(c, 1, 4, max_pages=4)
    slot, k = torch.zeros(1, 3, dtype=torch.int64, device=dev()), torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device=dev())
    bad = [lambda: swa.kv4_attention(c, q.half(), table, lens, workspace=ws), lambda: swa.kv4_attention(c, q, table.long(), lens, workspace=ws),
           lambda: swa.kv4_attention(c, q, table, lens, workspace=ws.cpu()), lambda: swa.kv4_attention(c.cpu(), q, table, lens, workspace=ws),
           lambda: swa.kv4_attention(c, q[:, :3].contiguous(), table, lens, workspace=ws),
           lambda: swa.kv4_attention(c, q, table, lens, workspace=ws[:256]), lambda: swa.kv4_attention(c, q, table, lens, window=-3, workspace=ws),
           lambda: swa.kv4_append(c, k, k, slot.int()), lambda: swa.kv4_append(c, k, k[:, :, :1], slot), lambda: swa.kv4_append(c, k, k, None),
           lambda: swa.kv4_read(c, slot[0]), lambda: swa.kv4_read(c, slot.cpu()), lambda: swa.kv4_read(c, slot, dtype=torch.float16),
           lambda: swa.kv4_plan(lens, lens, table, lens, lens, page=24, n_pages=4, n_tokens=1),
           lambda: swa.kv4_plan(lens, lens, table, lens, None, page=16, n_pages=4, n_tokens=1),
           lambda: swa.rope_tables(8, 24), lambda: swa.rope_tables(-1, 16), lambda: swa.rope_apply(q, None, swa.rope_tables(4, 64)),
           lambda: swa.rope_apply(k, None, swa.rope_tables(2, 64))]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, swa.SwaError)):
            f()
            print("call", i, "was taken")
    # a stream of its own, a raw handle, a row of tables as one tensor
    o = swa.kv4_attention(c, q, table, lens, workspace=ws, stream=torch.cuda.current_stream())
    p = swa.kv4_attention(c, q, table, lens, rope=torch.stack(swa.rope_tables(4, 64)), workspace=ws)
    assert o[0].shape == p[0].shape
    assert swa.rope_tables(0, 16)[0].shape == (0, 8)

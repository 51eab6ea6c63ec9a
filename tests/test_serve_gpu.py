"""GPU parity of the norm, the 4-bit projections and the drafted tokens' entry
points against the float64 oracle (oracle/serve.py), for both builds.

Bounds (a rounding is off by at most half a step: U = 2^-24 in fp32, 2^-8 in
bf16, 2^-11 in fp16, relative to the value):
  norm      h is one rounding of an fp32 sum: compared bit for bit. The sum of C
            squares is a tree of at most C / 32 + 16 additions in a row, half of
            whose relative error reaches rstd, with the root's 2 ulp and two
            products: (C / 64 + 16) U, and half a step of y. The e4m3 numbers are
            the oracle's, all of them.
  backward  the sum of C products likewise: see back_bounds.
  linear    products are exact; K additions in fp32, of which a product
            instruction may cut rather than round (2 U each): 2 K U of the sum of
            sizes, and half a step of y. bf16 calls of more than 32 rows meet weights
            rounded to bf16: 2^-8 of that sum more.
  tree      as the decode attention (a logit's products sum to at most 30 in
            absolute value; the query's two fp16 terms, norm and accumulation make it
            wrong by 8e-5): lse within 1e-4. In bf16 calls P is one bf16 term, 2^-8: o
            within 2 * 8e-5 + 2^-8 of the largest value (fp32 calls: 1.7e-4 of it),
            and half a step. The roundings of a row are many and independent, so
            the whole of o is also held to 2^-8 (P) + 2^-8 (o) + 1e-3 = 0.9 % in the
            2-norm.
"""

import numpy as np
import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from oracle import decode as dec
from oracle import serve
from test_decode_gpu import build_cache, f64, randn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = ["bf16", "fp32"]
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": U}


def dev():
    return torch.device("cuda:0")


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=dev())


# ---------------------------------------------------------------------------
# Norm
# ---------------------------------------------------------------------------

WIDTHS = [8, 64, 72, 768, 1000, 1024, 1032, 2048, 3080, 4096, 4104, 8192, 9000, 16384, 16392, 65536]
ROWS = {8: 77, 64: 9, 768: 300}


def norm_inputs(kind, C, rows, seed=0):
    x, a = (randn(seed + i, rows, C, dtype=DT[kind]) for i in range(2))
    return x, a, 1 + 0.1 * randn(seed + 2, C)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("add,gain,fp8", [(True, True, False), (False, False, False), (True, True, True), (False, False, True)])
def test_norm(kind, C, add, gain, fp8):
    rows = ROWS.get(C, 5)
    x, a, g = norm_inputs(kind, C, rows)
    a, g = a if add else None, g if gain else None
    r = swa.rms_norm(x.to(dev()), None if g is None else g.to(dev()), add=None if a is None else a.to(dev()), fp8=fp8)
    h = x if a is None else (x.float() + a.float()).to(x.dtype)
    assert torch.equal(r["h"].cpu(), h)
    gd = None if g is None else f64(g)
    y, rstd = serve.norm(f64(h), gd)
    tol = (C / 64 + 16) * U
    assert np.all(np.abs(f64(r["rstd"]) - rstd) <= tol * rstd)
    if fp8:
        n, s = serve.norm8(f64(h), gd)
        assert r["y"].dtype == torch.float8_e4m3fn
        assert np.array_equal(f64(r["y"].float()), n)
        assert np.all(np.abs(f64(r["scale"]) - s) <= tol * s)
    else:
        assert r["scale"] is None
        assert np.all(np.abs(f64(r["y"]) - y) <= (tol + HALF[kind]) * np.abs(y))


@pytest.mark.parametrize("kind", KINDS)
def test_norm_in_8_bits_at_borders(kind):
    # rows whose quotients lie on, or a last bit off, a border between two numbers: u 448 / top = 448 k / 2^j
    C, rows = 512, 64
    mids = (serve.round8(np.linspace(0.01, 448, 4000)))
    mids = np.unique(mids)
    mids = (mids[1:] + mids[:-1]) / 2
    x = torch.zeros(rows, C, dtype=torch.float64)
    for i in range(rows):
        top = 448.0 * 2.0 ** (i % 5 - 2)
        pick = torch.tensor(np.random.default_rng(i).choice(mids, C)) * top / 448.0
        step = 2.0 ** -23 if kind == "fp32" else 2.0 ** -7
        x[i] = pick * (1 + step * torch.tensor(np.random.default_rng(100 + i).integers(-1, 2, C)))
        x[i, i] = -top if i & 1 else top
    x = x.float().to(DT[kind])
    for g in (None, 1 + 0.25 * randn(5, C), torch.full((C,), 1.0 / 3.0)):
        r = swa.rms_norm(x.to(dev()), None if g is None else g.to(dev()), fp8=True)
        n, s = serve.norm8(f64(x), None if g is None else f64(g))
        assert np.array_equal(f64(r["y"].float()), n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [64, 2048, 20000])
@pytest.mark.parametrize("power,eps", [(100, 1e-6), (126, 1e-6), (-100, 0.0), (-120, 0.0), (-100, 1e-6), (-60, 1e-20), (-41, 1e-6)])
def test_norm_of_rows_near_the_ends_of_fp32(kind, C, power, eps):
    x = (randn(3, 4, C).clamp(-1.9, 1.9) * 2.0 ** power).to(DT[kind])
    h, tol = f64(x), (C / 64 + 16) * U
    y, rstd = serve.norm(h, None, eps)
    r = swa.rms_norm(x.to(dev()), eps=eps)
    assert np.all(np.abs(f64(r["rstd"]) - rstd) <= tol * rstd + 2.0 ** -149)
    assert np.all(np.abs(f64(r["y"]) - y) <= (tol + HALF[kind]) * np.abs(y) + 2.0 ** -133)
    r = swa.rms_norm(x.to(dev()), eps=eps, fp8=True)
    n, s = serve.norm8(h, None, eps)
    assert np.array_equal(f64(r["y"].float()), n)
    assert np.all(np.abs(f64(r["scale"]) - s) <= tol * s + 2.0 ** -149)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [64, 2048, 20000])
def test_norm_keeps_odd_rows_apart(kind, C):
    x = randn(4, 6, C, dtype=DT[kind])
    x[1, 7], x[2, 3], x[3] = float("nan"), float("inf"), 0.0
    r = swa.rms_norm(x.to(dev()))
    y = f64(r["y"])
    assert np.isnan(y[1]).all() and np.isnan(y[2, 3]) and not y[3].any()
    ok = [0, 4, 5]
    want = serve.norm(f64(x)[ok])[0]
    assert np.all(np.abs(y[ok] - want) <= ((C / 64 + 16) * U + HALF[kind]) * np.abs(want))
    r = swa.rms_norm(x.to(dev()), fp8=True)
    v = f64(r["y"].float()) * f64(r["scale"])[:, None]
    assert np.isnan(v[1:3]).all() and not v[3].any() and np.isfinite(v[ok]).all()
    # gains so small that 448 over the largest product would pass fp32's end
    r = swa.rms_norm(x[:1].to(dev()), torch.full((C,), 1e-38, device=dev()), fp8=True)
    assert not f64(r["y"].float()).any() and not f64(r["scale"]).any()


def test_norm_shapes_places_and_nothing():
    x, a, g = (t.to(dev()) for t in norm_inputs("bf16", 96, 30))
    want = swa.rms_norm(x, g, add=a)
    # leading dimensions
    r = swa.rms_norm(x.view(5, 2, 3, 96), g, add=a.view(5, 2, 3, 96))
    assert r["rstd"].shape == (5, 2, 3) and torch.equal(r["y"].view(30, 96), want["y"])
    # h over x; and through the C entry h over add, y over x
    x2 = x.clone()
    r = swa.rms_norm(x2, g, add=a, inplace=True)
    assert r["h"] is x2 and torch.equal(x2, want["h"]) and torch.equal(r["y"], want["y"])
    x2, a2 = x.clone(), a.clone()
    assert swa.swa_rms_norm(30, 96, 1e-6, x2, a2, g, a2, x2, None, None, None) == swa.SWA_OK
    assert torch.equal(a2, want["h"]) and torch.equal(x2, want["y"])
    # a row longer than registers hold, in place
    xl, al, gl = (t.to(dev()) for t in norm_inputs("bf16", 40000, 3))
    wl = swa.rms_norm(xl, gl, add=al)
    x2, a2 = xl.clone(), al.clone()
    assert swa.swa_rms_norm(3, 40000, 1e-6, x2, a2, gl, a2, x2, None, None, None) == swa.SWA_OK
    assert torch.equal(a2, wl["h"]) and torch.equal(x2, wl["y"])
    assert swa.rms_norm(x)["h"] is x
    r = swa.rms_norm(x[:0], g, add=a[:0], fp8=True)
    assert r["y"].shape == (0, 96) and r["scale"].shape == (0,)
    with pytest.raises(swa.SwaError):
        swa.rms_norm(torch.zeros(2, 60, device=dev()))
    with pytest.raises(ValueError):
        swa.rms_norm(x, g.cpu())


def back_bounds(h, rstd, dy, g, dh, dx, rows, C):
    """What fp32 may leave dx and dgain off by."""
    xh, d = np.abs(h) * rstd[:, None], np.abs(dy) * (1 if g is None else np.abs(g))
    mean = (xh * d).mean(-1, keepdims=True)
    bx = rstd[:, None] * (6 * U * d + xh * mean * (C / 32 + 24) * U) + 2 * U * (np.abs(dx) + (0 if dh is None else np.abs(dh)))
    return bx, (rows + 8) * U * (np.abs(dy) * xh).sum(0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("gain,add", [(True, True), (False, False)])
def test_norm_backward(kind, C, gain, add):
    rows = ROWS.get(C, 5)
    h, dh, g = norm_inputs(kind, C, rows, 20)
    dy = randn(23, rows, C, dtype=DT[kind])
    g, dh = g if gain else None, dh if add else None
    rstd = swa.rms_norm(h.to(dev()))["rstd"]
    r = swa.rms_norm_backward(h.to(dev()), rstd, dy.to(dev()), None if g is None else g.to(dev()),
                              dh=None if dh is None else dh.to(dev()))
    hd, rd, yd, gd, ed = f64(h), f64(rstd), f64(dy), None if g is None else f64(g), None if dh is None else f64(dh)
    dx, dg = serve.norm_backward(hd, rd, yd, gd, ed)
    bx, bg = back_bounds(hd, rd, yd, gd, ed, dx, rows, C)
    assert np.all(np.abs(f64(r["dx"]) - dx) <= bx + HALF[kind] * np.abs(dx))
    assert np.all(np.abs(f64(r["dgain"]) - dg) <= bg)
    only = swa.rms_norm_backward(h.to(dev()), rstd, dy.to(dev()), None if g is None else g.to(dev()),
                                 dh=None if dh is None else dh.to(dev()), need_gain=False)
    assert only["dgain"] is None and torch.equal(only["dx"], r["dx"])


@pytest.mark.parametrize("C", [96, 2048, 20000])
def test_norm_backward_by_differences_in_place_and_repeated(C):
    # the forward's own differences, in fp32 along random directions
    rows = 2000 if C == 96 else 700
    h, dy, g = norm_inputs("fp32", C, rows, 30)
    h, dy, g = h.to(dev()), dy.to(dev()), g.to(dev())
    f = swa.rms_norm(h, g)
    r = swa.rms_norm_backward(h, f["rstd"], dy, g)
    for x, grad, at in ((h, r["dx"], 0), (g, r["dgain"], 1)):
        e = randn(33 + at, *x.shape).to(dev())
        t = 2.0 ** -6
        up, down = ((swa.rms_norm(h + s * e, g) if at == 0 else swa.rms_norm(h, g + s * e))["y"] for s in (t, -t))
        got = ((up.double() - down.double()) * dy).sum().item() / (2 * t)
        want = (grad.double() * e).sum().item()
        # the third derivative's t^2 / 6 and the fp32 roundings of y over t, as random signs over all entries
        size = (dy.double().square().sum().sqrt()).item()
        assert abs(got - want) <= size * (t * t + 8 * U / t)
    ws = torch.full((swa.swa_rms_norm_workspace_size(rows, C, "fp32"),), 255, dtype=torch.uint8, device=dev())
    for _ in range(3):
        again = swa.rms_norm_backward(h, f["rstd"], dy, g, workspace=ws)
        assert torch.equal(again["dx"], r["dx"]) and torch.equal(again["dgain"], r["dgain"])
    for name in ("dy", "h"):
        h2, d2 = h.clone(), dy.clone()
        out = d2 if name == "dy" else h2
        dg = torch.empty(C, device=dev())
        assert swa.swa_rms_norm_bwd(rows, C, h2, f["rstd"], g, d2, None, out, dg, ws) == swa.SWA_OK
        assert torch.equal(out, r["dx"]) and torch.equal(dg, r["dgain"])
    empty = swa.rms_norm_backward(h[:0], f["rstd"][:0], dy[:0], g)
    assert empty["dx"].shape == (0, C) and not empty["dgain"].any()


# ---------------------------------------------------------------------------
# 4-bit projections
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,K", [(1, 8), (16, 64), (37, 200), (130, 768)])
def test_w4_pack_and_unpack(kind, N, K):
    w = randn(40, N, K, dtype=DT[kind])
    w[0, :8] = 0.0
    if K > 64:
        w[N // 2, 64:128] = 0.0
    if K > 128:
        w[-1, 128:] *= 1e-37
    n, s = serve.w4_quantise(f64(w))
    w4 = swa.w4_pack(w.to(dev()))
    assert np.array_equal(w4.cpu().numpy(), serve.w4_tiles(n, s))
    back = swa.w4_unpack(w4, N, K, dtype=DT[kind])
    want = serve.w4_values(w4.cpu().numpy(), N, K)
    assert np.array_equal(f64(back), want if kind == "fp32" else dec.bf16(want))


@pytest.mark.parametrize("kind", KINDS)
def test_w4_numbers_at_borders(kind):
    # entries on and beside the borders (n - 7.5) s of a step that the largest entry gives
    rows = []
    for i in range(48):
        top = float(torch.tensor(1.0 + i / 7.0).to(DT[kind]))
        s = dec.bf16(np.float64(np.float32(top) / np.float32(7.0)))
        b = (np.arange(16) - 7.5) * s
        row = np.concatenate([[top], b, np.nextafter(b.astype(np.float32), np.float32(9e9)), np.nextafter(b.astype(np.float32), np.float32(-9e9)),
                              -b[:15]])
        rows.append(np.clip(row, -top, top))
    w = torch.tensor(np.array(rows), dtype=torch.float64).float().to(DT[kind])
    assert w.shape[1] == 64
    n, s = serve.w4_quantise(f64(w))
    assert np.array_equal(swa.w4_pack(w.to(dev())).cpu().numpy(), serve.w4_tiles(n, s))


def test_w4_group_that_is_not_finite():
    w = randn(41, 20, 136)
    w[3, 70], w[17, 0] = float("inf"), float("nan")
    v = f64(swa.w4_unpack(swa.w4_pack(w.to(dev())), 20, 136, dtype=torch.float32))
    assert np.isnan(v[3, 64:128]).all() and np.isnan(v[17, :64]).all()
    v[3, 64:128] = v[17, :64] = 0.0
    assert np.isfinite(v).all()


def random_w4(seed, N, K):
    g = torch.Generator().manual_seed(seed)
    P, Q = -(-N // 16), -(-K // 64)
    w = torch.randint(0, 256, (P, Q, 544), generator=g, dtype=torch.uint8)
    s = (torch.rand(P, Q, 16, generator=g) * 0.2 + 0.05) * torch.where(torch.rand(P, Q, 16, generator=g) < 0.5, -1.0, 1.0)
    w[..., 512:].view(torch.bfloat16).copy_(s)
    return w


def linear_case(kind, M, N, K, x8=False, add=False, seed=50):
    w4 = random_w4(seed, N, K)
    x = randn(seed + 1, M, K)
    scale = None
    if x8:
        scale = x.abs().amax(-1) / 448
        x = (x / scale[:, None]).to(torch.float8_e4m3fn)
    else:
        x = x.to(DT[kind])
    r = randn(seed + 2, M, N, dtype=DT[kind]) if add else None
    xd = f64(x.float()) * (1 if scale is None else f64(scale)[:, None])
    w = serve.w4_values(w4.numpy(), N, K)
    want = xd @ w.T + (0 if r is None else f64(r))
    size = np.abs(xd) @ np.abs(w).T + (0 if r is None else np.abs(f64(r)))
    return w4, x, scale, r, want, size


def check_linear(y, kind, want, size, M, K, x8):
    tol = 2 * (K + 8) * U * size + HALF[kind] * np.abs(want)
    if kind == "bf16" and M > 32:
        tol = tol + 2.0 ** -8 * size
    err = np.abs(f64(y) - want)
    assert np.all(err <= tol), float((err - tol).max())
    assert np.linalg.norm(err) <= (1e-2 if kind == "bf16" else 2e-6) * np.linalg.norm(want)


LINEAR = [(1, 16, 64), (1, 1, 8), (2, 7, 72), (3, 40, 200), (8, 128, 768), (9, 130, 776), (15, 33, 1000), (16, 64, 64), (17, 100, 136),
          (24, 300, 512), (33, 129, 264), (64, 256, 1024), (65, 48, 72), (100, 500, 640), (129, 260, 392), (260, 140, 328), (300, 1000, 256)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(kind, x8, M, N, K):
    for add in (False, True):
        w4, x, scale, r, want, size = linear_case(kind, M, N, K, x8, add)
        y = swa.w4_linear(x.to(dev()), w4.to(dev()), out_features=N, scale=None if scale is None else scale.to(dev()),
                          add=None if r is None else r.to(dev()), dtype=DT[kind])
        check_linear(y, kind, want, size, M, K, x8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("x8", [False, True])
def test_linear_of_a_wide_layer_repeats_its_bits(kind, x8):
    for M in (1, 5, 20, 70):
        w4, x, scale, r, want, size = linear_case(kind, M, 2048, 4096, x8, True, 60)
        a = [t if t is None else t.to(dev()) for t in (x, w4, scale, r)]
        ys = [swa.w4_linear(a[0], a[1], scale=a[2], add=a[3], dtype=DT[kind]) for _ in range(3)]
        check_linear(ys[0], kind, want, size, M, 4096, x8)
        assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
        y = a[3].clone()                                # onto the residual
        assert swa.w4_linear(a[0], a[1], scale=a[2], add=y, dtype=DT[kind], out=y) is y and torch.equal(y, ys[0])


@pytest.mark.parametrize("kind", KINDS)
def test_a_row_of_a_batch_does_not_see_the_others(kind):
    # a NaN, an infinity and huge entries stay in their rows, and in the outputs of their weights
    for M in (4, 40, 200):
        w4, x, _, _, want, size = linear_case(kind, M, 64, 256, seed=70)
        x[1, 5], x[2, 9], x[3] = float("nan"), float("inf"), x[3] * 1e30
        want[3], size[3] = (f64(x[3:4]) @ serve.w4_values(w4.numpy(), 64, 256).T)[0], size[3] * 1e30
        y = swa.w4_linear(x.to(dev()), w4.to(dev()))
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
        keep = [i for i in range(M) if i not in (1, 2)]
        err = np.abs(f64(y)[keep] - want[keep])
        assert np.all(err <= 2 * 264 * U * size[keep] + (2.0 ** -7 if kind == "bf16" else U) * size[keep])


def test_linear_takes_shapes_and_nothing():
    w4 = random_w4(80, 48, 128).to(dev())
    x = randn(81, 2, 3, 128, dtype=torch.bfloat16).to(dev())
    y = swa.w4_linear(x, w4)
    assert y.shape == (2, 3, 48) and torch.equal(y.view(6, 48), swa.w4_linear(x.view(6, 128), w4))
    assert swa.w4_linear(x[:0], w4).shape == (0, 3, 48)
    assert torch.equal(swa.w4_linear(x, w4, out_features=41).reshape(6, 41), y.view(6, 48)[:, :41])
    one = swa.w4_linear(x[0, 0], w4)
    assert one.shape == (48,) and torch.equal(one, y[0, 0])


def test_norm_in_8_bits_feeds_the_projection():
    x, a, g = (t.to(dev()) for t in norm_inputs("bf16", 256, 12, 90))
    w4 = random_w4(91, 80, 256)
    r = swa.rms_norm(x, g, add=a, fp8=True)
    y = swa.w4_linear(r["y"], w4.to(dev()), scale=r["scale"])
    xd, w = f64(r["y"].float()) * f64(r["scale"])[:, None], serve.w4_values(w4.numpy(), 80, 256)
    check_linear(y, "bf16", xd @ w.T, np.abs(xd) @ np.abs(w).T, 12, 256, True)


# ---------------------------------------------------------------------------
# Drafted tokens
# ---------------------------------------------------------------------------

def random_parents(n, seed):
    g = np.random.default_rng(seed)
    return [-1 if i == 0 or g.random() < 0.1 else int(g.integers(max(0, i - 5), i)) for i in range(n)]


def flat(new, pad=0):
    cu = np.concatenate([[0], np.cumsum(new)])
    return cu, int(cu[-1]) + pad


@pytest.mark.parametrize("new,pad", [([1], 0), ([0, 3, 64, 0, 17], 5), ([64] * 9, 0), ([0, 0], 3), (list(range(1, 40)), 1)])
def test_tree(new, pad):
    cu, N = flat(new, pad)
    lens = [n + 7 * i for i, n in enumerate(new)]
    parent = np.full(N, 5)
    for b, n in enumerate(new):
        parent[cu[b]:cu[b + 1]] = random_parents(n, b)
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    pos, seen = swa.kv4_tree(i32(*parent), i32(*cu), i32(*lens), max_new=64, workspace=ws)
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK
    want_p, want_s = np.zeros(N, dtype=np.int64), np.zeros(N, dtype=np.uint64)
    for b, n in enumerate(new):
        p, s = serve.tree(list(parent[cu[b]:cu[b + 1]]), lens[b] - n)
        want_p[cu[b]:cu[b + 1]], want_s[cu[b]:cu[b + 1]] = p, s
    assert np.array_equal(pos.cpu().numpy(), want_p)
    assert np.array_equal(seen.cpu().numpy().view(np.uint64), want_s)


def test_tree_refuses_on_the_device():
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())

    def run(parent, cu, lens, max_new=8, n=None):
        pos, seen = swa.kv4_tree(i32(*parent), i32(*cu), i32(*lens), max_new=max_new, workspace=ws)
        return swa.swa_attn_check_status(ws), pos.tolist(), seen.tolist()
    bad = swa.SWA_ERR_DEVICE_CHECK
    # a parent that is not in front: the token and those below it
    assert run([-1, 1, 1, 0], [0, 4], [10]) == (bad, [6, 0, 0, 7], [1, 0, 0, 9])
    assert run([-1, -2, 1, 0], [0, 4], [10]) == (bad, [6, 0, 0, 7], [1, 0, 0, 9])
    assert run([2 ** 31 - 1, -2 ** 31], [0, 2], [10]) == (bad, [0, 0], [0, 0])
    # too many tokens, more than the request holds, a negative length
    assert run([-1, 0, 1], [0, 3], [10], max_new=2) == (bad, [0] * 3, [0] * 3)
    assert run([-1, 0, -1], [0, 2, 3], [1, 1]) == (bad, [0, 0, 0], [0, 0, 1])
    assert run([-1, -1], [0, 1, 2], [-4, 2 ** 31 - 1]) == (bad, [0, 2 ** 31 - 2], [0, 1])
    # rows that lie outside: not touched, so only the status is looked at
    for cu in ([0, 9], [-1, 2], [2, 1], [0, -5]):
        assert run([-1, 0], cu, [10])[0] == bad
    assert run([-1, 0], [0, 2], [2]) == (swa.SWA_OK, [0, 1], [1, 3])


def tree_case(kind, lens, new, Hq, Hkv, d, page, window, rot, inter, seed=1, pad=3, gain=True, scale=0.0, workspace=None,
              parents=None, stream=None):
    """Runs the attention of random trees and holds it to the oracle; returns o, lse."""
    cache, table, rows = build_cache(lens, Hkv, d, page, seed)
    cu, N = flat(new, pad)
    q = randn(seed + 1, N, Hq, d, dtype=DT[kind])
    gq = 1 + 0.1 * randn(seed + 2, d) if gain else None
    tabs = None if not rot else tuple(torch.tensor(x, dtype=torch.float32) for x in dec.rope_tables(max(lens + [1]), rot))
    trees = [serve.tree(random_parents(n, seed + b) if parents is None else parents(n), m - n) for b, (n, m) in enumerate(zip(new, lens))]
    pos = np.concatenate([t[0] for t in trees] + [[-7] * pad]).astype(np.int64)
    seen = np.array([s for t in trees for s in t[1]] + [0] * pad, dtype=np.uint64).view(np.int64)
    cd = cache.to(dev())
    ws = workspace if workspace is not None else swa.new_kv4_workspace(cd, len(lens), Hq, max_pages=table.shape[1], kind=kind)
    o, lse = swa.kv4_tree_attention(cd, q.to(dev()), table.to(dev()), i32(*lens), i32(*cu), i32(*pos), torch.tensor(seen, device=dev()),
                                    max_new=max(new + [1]), rope=None if tabs is None else tuple(t.to(dev()) for t in tabs),
                                    interleaved=inter, gq=None if gq is None else gq.to(dev()), window=window, softmax_scale=scale,
                                    workspace=ws, stream=stream)
    if stream is not None:
        stream.synchronize()
    assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
    assert torch.equal(cd.cpu(), cache)
    od, ld = f64(o), f64(lse)
    total, off = 0.0, 0.0
    for b, (n, m) in enumerate(zip(new, lens)):
        at = slice(cu[b], cu[b + 1])
        kw = {} if tabs is None else dict(cos=f64(tabs[0]), sin=f64(tabs[1]), interleaved=inter)
        ro, rl = serve.tree_attend(f64(q)[at], *rows[b], *trees[b], window=window, gq=None if gq is None else f64(gq), scale=scale, **kw)
        if n == 0:
            continue
        top = np.abs(rows[b][1]).max()
        tol_l, tol_o = 1e-4, (1.7e-4 + (2.0 ** -8 if kind == "bf16" else 0)) * top
        fine = np.isfinite(rl)
        assert np.array_equal(ld[at] == -np.inf, ~fine)
        assert np.all(np.abs(ld[at][fine] - rl[fine]) <= tol_l), float(np.abs(ld[at][fine] - rl[fine]).max())
        err = np.abs(od[at] - ro)
        assert np.all(err <= tol_o + HALF[kind] * np.abs(ro)), float(err.max())
        total, off = total + (ro ** 2).sum(), off + (err ** 2).sum()
    assert off <= (9e-3 if kind == "bf16" else 1e-5) ** 2 * total, (off / total) ** 0.5
    assert not od[cu[-1]:].any() and np.all(ld[cu[-1]:] == -np.inf)
    return o, lse


SHORT = [1, 0, 2, 15, 16, 17, 31, 32, 33, 47, 64, 65, 100, 127, 129, 200]
FEW = [1, 0, 2, 1, 3, 4, 2, 4, 1, 3, 4, 2, 1, 4, 4, 3]
TREES = [  # lens, new, Hq, Hkv, d, page, window, rot, interleaved
    (SHORT, FEW, 4, 2, 128, 16, -1, 128, False),
    (SHORT, FEW, 2, 1, 64, 48, -1, 64, False),
    (SHORT, FEW, 6, 3, 128, 64, 40, 128, False),
    (SHORT, FEW, 3, 3, 64, 32, 0, 32, True),
    (SHORT, FEW, 9, 1, 64, 32, 2, 48, True),
    (SHORT, FEW, 17, 1, 128, 16, 1, 64, True),
    ([8, 40, 33, 100], [8, 8, 5, 7], 4, 1, 128, 16, -1, 128, False),             # 32 rows
    ([17, 64, 90], [17, 13, 16], 2, 1, 64, 32, 10, 16, True),                    # 34 rows
    ([16, 70, 200], [16, 15, 1], 4, 1, 128, 32, -1, 96, False),                  # 64 rows
    ([64, 300, 65], [64, 64, 63], 1, 1, 128, 64, -1, 0, False),
    ([70, 128], [64, 33], 6, 3, 64, 16, 20, 64, False),                          # 128 rows, two groups
    ([1500, 3, 777, 0], [6, 3, 5, 0], 4, 1, 128, 64, -1, 128, False),
    ([2500], [11], 2, 2, 64, 16, -1, 64, False),
    ([2048, 2049, 40], [20, 24, 24], 4, 2, 128, 256, 1000, 128, False),
    ([3000, 2999], [40, 33], 2, 1, 128, 64, 2000, 64, True),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,Hq,Hkv,d,page,window,rot,inter", TREES)
def test_tree_attention(kind, lens, new, Hq, Hkv, d, page, window, rot, inter):
    tree_case(kind, lens, new, Hq, Hkv, d, page, window, rot, inter)


@pytest.mark.parametrize("kind", KINDS)
def test_tree_attention_without_gain_and_with_a_scale(kind):
    tree_case(kind, [70, 5], [6, 5], 4, 2, 128, 32, -1, 0, False, gain=False, scale=0.05)
    tree_case(kind, [70, 33], [30, 20], 2, 2, 64, 16, -1, 64, False, gain=False)


@pytest.mark.parametrize("kind", KINDS)
def test_one_drafted_token_is_the_decode_attention(kind):
    lens, Hq, Hkv, d, page = [5, 100, 63, 2000], 4, 2, 128, 32
    cache, table, _ = build_cache(lens, Hkv, d, page, 9)
    q, cd, td = randn(10, 4, Hq, d, dtype=DT[kind]).to(dev()), cache.to(dev()), table.to(dev())
    rope = swa.rope_tables(2000, d)
    o1, l1 = swa.kv4_attention(cd, q, td, i32(*lens), rope=rope, window=300)
    pos, seen = swa.kv4_tree(i32(-1, -1, -1, -1), i32(0, 1, 2, 3, 4), i32(*lens), max_new=1)
    o2, l2 = swa.kv4_tree_attention(cd, q, td, i32(*lens), i32(0, 1, 2, 3, 4), pos, seen, max_new=1, rope=rope, window=300)
    assert (l1 - l2).abs().max().item() <= 2e-4
    assert (o1.double() - o2.double()).norm() <= (1e-2 if kind == "bf16" else 1e-5) * o1.double().norm()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,T", [(2, 4), (4, 8), (4, 16)])
def test_what_a_token_does_not_see_changes_nothing(kind, Hq, T):
    # NaN in the cached rows of one branch: the tokens of the others give the same bits as without
    d, page, n = 128, 16, 150
    cache, table, _ = build_cache([n], 1, d, page, 11)
    parent = [-1] + [0 if i < 3 else i - 2 for i in range(1, T)]           # two branches
    pos, seen = serve.tree(parent, n - T)
    q, cu = randn(12, T, Hq, d, dtype=DT[kind]).to(dev()), i32(0, T)
    args = (table.to(dev()), i32(n), cu, i32(*pos), torch.tensor(seen, device=dev()))
    want = swa.kv4_tree_attention(cache.to(dev()), q, *args, max_new=T)
    assert torch.isfinite(want[0]).all()
    t = n - T + 2                                                       # the second branch's first token
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, 2, 2)
    sc[int(table[0, t // page]), :, t % page // 16, :, t % 16] = float("nan")
    got = swa.kv4_tree_attention(cache.to(dev()), q, *args, max_new=T)
    for i in range(T):
        if seen[i] >> 2 & 1:
            assert torch.isnan(got[0][i]).any()
        else:
            assert torch.equal(got[0][i], want[0][i]) and torch.equal(got[1][i], want[1][i])
    # the same in the context, in front of the later tokens' window
    cache, table, _ = build_cache([n], 1, d, page, 11)
    pos, seen = serve.tree(list(range(-1, T - 1)), n - T)
    args = (table.to(dev()), i32(n), cu, i32(*pos), torch.tensor(seen, device=dev()))
    want = swa.kv4_tree_attention(cache.to(dev()), q, *args, max_new=T, window=60)
    t = n - T - 60
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(*cache.shape[:3], 2, 16, 2, 2)
    sc[int(table[0, t // page]), :, t % page // 16, :, t % 16] = float("nan")
    got = swa.kv4_tree_attention(cache.to(dev()), q, *args, max_new=T, window=60)
    assert torch.isnan(got[0][0]).any() and torch.equal(got[0][1:], want[0][1:]) and torch.equal(got[1][1:], want[1][1:])


@pytest.mark.parametrize("kind", KINDS)
def test_tree_attention_reports_what_it_leaves_out(kind):
    d, page = 64, 16
    cache, table, _ = build_cache([40, 50], 1, d, page, 13)
    cd, td = cache.to(dev()), table.to(dev())
    ws = swa.new_kv4_workspace(cd, 2, 2, max_pages=td.shape[1], kind=kind)
    q = randn(14, 6, 2, d, dtype=DT[kind]).to(dev())
    rope = tuple(t.to(dev()) for t in swa.rope_tables(50, d))

    def run(lens=(40, 50), cu=(0, 3, 6), pos=(37, 38, 39, 47, 48, 49), seen=(1, 3, 7) * 2, table=td, max_new=4, rope=rope):
        o, lse = swa.kv4_tree_attention(cd, q, table, i32(*lens), i32(*cu), i32(*pos), torch.tensor(seen, device=dev()),
                                        max_new=max_new, rope=rope, workspace=ws)
        return swa.swa_attn_check_status(ws, kind=kind), o, lse
    bad = swa.SWA_ERR_DEVICE_CHECK
    st, o, lse = run()
    assert st == swa.SWA_OK and torch.isfinite(lse).all()

    def hidden(r, rows):
        assert r[0] == bad
        for i in range(6):
            if i in rows:
                assert not r[1][i].any() and torch.isinf(r[2][i]).all()
            else:
                assert torch.equal(r[1][i], o[i]) and torch.equal(r[2][i], lse[i])
    hidden(run(pos=(37, 38, 36, 47, 48, 49)), [2])                          # in front of the context's end
    hidden(run(pos=(37, 38, 39, 47, 48, 50)), [5])                          # outside the tables
    hidden(run(lens=(-3, 50)), [0, 1, 2])
    hidden(run(lens=(2, 50)), [0, 1, 2])                                    # more drafted than cached
    hidden(run(lens=(page * td.shape[1] + 1, 50)), [0, 1, 2])
    hidden(run(max_new=2), [0, 1, 2, 3, 4, 5])
    st, o2, l2 = run(seen=(1, 3, 0, 1, 3, 7))                                 # sees nothing: no error
    assert st == swa.SWA_OK and not o2[2].any() and torch.isinf(l2[2]).all() and torch.equal(o2[3:], o[3:])
    st, o2, l2 = run(seen=(1, 3, 7 | 1 << 3 | 1 << 63 - 1, 1, 3, 7))           # bits behind the last token
    assert st == swa.SWA_OK and torch.equal(o2, o)
    for page_id in (-5, cd.shape[0]):
        t2 = td.clone()
        t2[0, 1] = page_id
        st, o2, _ = run(table=t2)
        assert st == bad and torch.isfinite(o2[:3]).all() and torch.equal(o2[3:], o[3:])
    for cu in ((0, 9, 6), (-1, 3, 6), (4, 3, 6), (0, 3, 7)):
        assert run(cu=cu)[0] == bad
    assert run()[0] == swa.SWA_OK


def test_tree_of_long_requests_repeats_its_bits():
    d, page, n = 128, 64, 8000
    n_pages = n // page + 2
    g = torch.Generator().manual_seed(15)
    cache = torch.randint(0, 256, (n_pages, 2, page // 16, 18 * d), generator=g, dtype=torch.uint8)
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc[..., 0::2] = 0.2
    sc[..., 1::2] = (0.2 * randn(16, *sc[..., 1::2].shape)).bfloat16()
    cache = cache.to(dev())
    table = torch.randperm(n_pages, generator=g)[None].int().to(dev())
    slot = (table[0].long()[:, None] * page + torch.arange(page, device=dev())).view(1, -1)[:, :n].contiguous()
    k, v = (x[0].double().cpu().numpy() for x in swa.kv4_read(cache, slot, dtype=torch.float32))
    for T in (3, 8, 20):
        pos, seen = serve.tree(random_parents(T, T), n - T)
        q = randn(17, T, 4, d, dtype=torch.bfloat16).to(dev())
        ws = swa.new_kv4_workspace(cache, 1, 4, max_pages=n_pages)
        for w in (-1, 5000):
            runs = [swa.kv4_tree_attention(cache, q, table, i32(n), i32(0, T), i32(*pos), torch.tensor(seen, device=dev()), max_new=T,
                                           window=w, workspace=ws) for _ in range(4)]
            for o, lse in runs[1:]:
                assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
            ro, rl = serve.tree_attend(f64(q), k, v, pos, seen, window=w)
            assert np.abs(f64(runs[0][1]) - rl).max() <= 1e-4
            assert np.linalg.norm(f64(runs[0][0]) - ro) <= 9e-3 * np.linalg.norm(ro)


def test_one_workspace_serves_both_attentions():
    ws = torch.full((swa.swa_kv4_workspace_size(swa.make_params(1, 1, 4, 2, 128), 64, 4),), 255, dtype=torch.uint8, device=dev())
    assert swa.swa_kv4_workspace_init(ws) == swa.SWA_OK
    from test_decode_gpu import check_attention
    for _ in range(2):
        tree_case("bf16", [3000, 2900], [9, 4], 4, 2, 128, 64, -1, 128, False, workspace=ws)
        check_attention("bf16", [3000, 2900], 4, 2, 128, 64, workspace=ws, seed=10)
        tree_case("bf16", [30] * 100, [7] * 100, 4, 2, 128, 16, -1, 0, False, workspace=ws)
        check_attention("bf16", [30] * 300, 4, 2, 128, 16, workspace=ws, seed=11)
        tree_case("bf16", [1800], [64], 9, 1, 64, 32, -1, 64, True, workspace=ws)


@pytest.mark.parametrize("kind", KINDS)
def test_tree_waits_that_run_out_are_reported_and_the_workspace_stays_usable(kind):
    # a limit of 1 ns, on requests whose 150 MB all come from memory while another stream keeps the memory busy: the
    # copies all land, only later. The arithmetic of many rows hides most of them, so that a call may well get through
    # in time: tries until one has not.
    d, page, n, Hkv, Hq, B = 128, 64, 8192, 2, 4, 64
    per = n // page
    cache = torch.randint(0, 256, (B * per, Hkv, page // 16, 18 * d), dtype=torch.uint8, device=dev())
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc[..., 0::2], sc[..., 1::2] = 0.2, 0.1
    table = torch.arange(B * per, dtype=torch.int32, device=dev()).view(B, per)
    lens = torch.full((B,), n, dtype=torch.int32, device=dev())
    side, big = torch.cuda.Stream(), [torch.zeros(1 << 28, device=dev()) for _ in range(2)]
    ran_out = 0
    for T in (2, 16, 32):
        cu = torch.arange(B + 1, dtype=torch.int32, device=dev()) * T
        parent = torch.arange(-1, T - 1, dtype=torch.int32, device=dev()).repeat(B)
        pos, seen = swa.kv4_tree(parent, cu, lens, max_new=T)
        q = randn(6, B * T, Hq, d, dtype=DT[kind]).to(dev())
        ws = swa.new_kv4_workspace(cache, B, Hq, max_pages=per, kind=kind)
        want = swa.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new=T, workspace=ws)
        assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
        p, c = swa.make_params(B, 1, Hq, Hkv, d), swa.swa_kv4_cache(cache.data_ptr(), B * per, page)
        o, lse = torch.empty_like(q), torch.empty(B * T, Hq, device=dev())
        short = swa.make_extras(wait_limit_ns=1)
        for _ in range(20):
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                for _ in range(3):
                    big[0].copy_(big[1])
            assert swa.swa_kv4_tree_attn(p, short, c, None, B * T, T, q, None, table, per, lens, cu, pos, seen, o, lse, ws) == swa.SWA_OK
            st = swa.swa_attn_check_status(ws, kind=kind)
            assert st in (swa.SWA_OK, swa.SWA_ERR_TIMEOUT)
            assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK      # read and cleared
            got = swa.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new=T, workspace=ws)
            assert swa.swa_attn_check_status(ws, kind=kind) == swa.SWA_OK
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            if st == swa.SWA_ERR_TIMEOUT:
                ran_out += 1
                break
    assert ran_out


# ---------------------------------------------------------------------------
# Move
# ---------------------------------------------------------------------------

def rows_at(cache, page, slots):
    """Each slot's bytes of every head, as the oracle reads them."""
    c = cache.numpy()
    return [[dec.read_row(c, page, s, h) for h in range(c.shape[1])] for s in slots]


@pytest.mark.parametrize("d,Hkv,page", [(64, 1, 16), (128, 3, 48)])
def test_move(d, Hkv, page):
    n_pages, T = 9, 64
    g = torch.Generator().manual_seed(18)
    cache = torch.randint(0, 256, (n_pages, Hkv, page // 16, 18 * d), generator=g, dtype=torch.uint8)
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc.copy_(torch.randn(sc.shape, generator=g))
    slots = torch.randperm(n_pages * page, generator=g)
    # row 0: chains, cycles and places that are both source and target; rows 1, 2: apart from it; skips among them
    mine = slots[:70].tolist()
    src, dst = torch.full((3, T), -1, dtype=torch.int64), torch.full((3, T), -1, dtype=torch.int64)
    src[0, :40] = torch.tensor(mine[:40])
    dst[0, :40] = torch.tensor(mine[1:40] + mine[:1])
    src[1, :3], dst[1, :3] = torch.tensor(mine[40:43]), torch.tensor([mine[43], -1, mine[44]])
    src[2, 5:9], dst[2, 5:9] = torch.tensor([mine[50], -1, mine[51], mine[52]]), torch.tensor([mine[53], mine[54], mine[51], mine[55]])
    before = {s: rows_at(cache, page, [s])[0] for s in mine}
    cd = cache.to(dev())
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    swa.kv4_move(cd, src.to(dev()), dst.to(dev()), workspace=ws)
    assert swa.swa_attn_check_status(ws) == swa.SWA_OK
    got = cd.cpu()
    moved = {int(b): int(a) for a, b in zip(src.flatten(), dst.flatten()) if a >= 0 and b >= 0}
    for s in mine:
        now, then = rows_at(got, page, [s])[0], before[moved.get(s, s)]
        for x, y in zip(now, then):
            assert all(np.array_equal(u, v) for u, v in zip(x, y))
    # back again row 0's cycle, and the places that no pair wrote are as they were
    swa.kv4_move(cd, dst[:1].contiguous().to(dev()), src[:1].contiguous().to(dev()))
    back = cd.cpu()
    for s in range(n_pages * page):
        if s in moved and s not in mine[:40]:
            continue
        for x, y in zip(rows_at(back, page, [s])[0], rows_at(cache, page, [s])[0]):
            assert all(np.array_equal(u, v) for u, v in zip(x, y))


def test_move_refuses_on_the_device():
    cache = torch.randint(0, 256, (2, 1, 1, 18 * 64), dtype=torch.uint8, device=dev())
    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    for src, dst in ((32, 0), (0, 32), (-2, 0), (0, -2), (2 ** 62, 1), (1, 2 ** 62)):
        c = cache.clone()
        swa.kv4_move(c, torch.tensor([[src, 3]], device=dev()), torch.tensor([[dst, 3]], device=dev()), workspace=ws)
        assert swa.swa_attn_check_status(ws) == swa.SWA_ERR_DEVICE_CHECK
        assert torch.equal(c, cache)
    swa.kv4_move(cache, torch.zeros(0, 4, dtype=torch.int64, device=dev()), torch.zeros(0, 4, dtype=torch.int64, device=dev()))
    with pytest.raises(swa.SwaError):
        swa.kv4_move(cache, torch.zeros(1, 65, dtype=torch.int64, device=dev()), torch.zeros(1, 65, dtype=torch.int64, device=dev()))

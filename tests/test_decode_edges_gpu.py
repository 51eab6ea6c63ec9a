"""The rotary and decode calls where their ranges end, for both builds:
infinities and NaN beside rows that are settled in 64 bits, rows too large
for fp32 squares, more tokens than a grid dimension holds, lengths
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
from test_decode_gpu import (DT, EPS, HALF, U, build_cache, check_held, dev, f64, gen, numbers_of, randn,
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


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_more_tokens_than_a_grid_dimension_holds(kind):
    # tokens of a step as n rows of one token, as a plan gives them, are the
    # same tokens as one row of n
    n, Hkv, d, page = 40001, 3, 64, 32
    n_pages = -(-n // page)
    k, v = (randn(i, n, 1, Hkv, d, dtype=DT[kind]).to(dev()) for i in (1, 2))
    slot = torch.randperm(n_pages * page, generator=gen(3))[:n].view(n, 1).to(dev())
    pos = torch.randint(0, 50, (n, 1), generator=gen(4), dtype=torch.int32).to(dev())
    rope = swa.rope_tables(50, d)
    got, want = (torch.zeros(n_pages, Hkv, page // 16, 18 * d, dtype=torch.uint8, device=dev()) for _ in range(2))
    swa.kv4_append(got, k, v, slot, pos=pos, rope=rope)
    swa.kv4_append(want, k.view(1, n, Hkv, d), v.view(1, n, Hkv, d), slot.view(1, n), pos=pos.view(1, n), rope=rope)
    assert torch.equal(got, want) and want.any()
    a, b = swa.kv4_read(got, slot, dtype=DT[kind]), swa.kv4_read(got, slot.view(1, n), dtype=DT[kind])
    for x, y in zip(a, b):
        assert x.shape == (n, 1, Hkv, d) and torch.equal(x.view(-1), y.view(-1))
    a = swa.rope_apply(k, v, rope, pos=pos)
    b = swa.rope_apply(k.view(1, n, Hkv, d), v.view(1, n, Hkv, d), rope, pos=pos.view(1, n))
    for x, y in zip(a, b):
        assert torch.equal(x.view(-1), y.view(-1))
    # many heads of few tokens
    q = randn(5, 2, 1, 40000, d, dtype=DT[kind]).to(dev())
    x, _ = swa.rope_apply(q, None, rope, pos=pos[:2])
    y, _ = swa.rope_apply(q.view(2, 20000, 2, d), None, rope, pos=pos[:2].expand(2, 20000).contiguous())
    assert torch.equal(x.view(-1), y.view(-1))


def test_plan_of_lengths_near_the_end_of_32_bits():
    # pages that are no power of two: the length rounded up to whole pages
    # passes 2^31 although the table row ends below it
    for page, width, lens, new in ((192, 11184810, [2147483500, 0], [10, 5]), (16000, 134217, [2147471997, 15999], [1, 2]),
                                   (144, 14913080, [2147483517, 2147483376], [3, 100])):
        n_pages, n_tokens = 12, sum(new) + 1
        table = np.full((2, width), -1, np.int32)
        for b, n in enumerate(lens):
            table[b, max(-(-n // page) - 2, 0):-(-n // page)] = 3 + b
        free, head = np.array([7, 8, 9], np.int32), 1
        ref = dec.plan(np.array(lens, np.int64), np.array(new, np.int64), table, free, head, page, n_pages, n_tokens)
        assert ref["refused"] == 0
        t = torch.tensor(table, device=dev())
        ws = torch.zeros(256, dtype=torch.uint8, device=dev())
        out = swa.kv4_plan(i32(*lens), i32(*new), t, i32(*free.tolist()), i32(head), page=page, n_pages=n_pages, n_tokens=n_tokens,
                           workspace=ws)
        assert swa.swa_attn_check_status(ws) == swa.SWA_OK
        assert np.array_equal(t.cpu().numpy(), ref["table"])
        for x in ("slot", "pos", "row", "cu", "lens"):
            np.testing.assert_array_equal(out[x].cpu().numpy(), ref[x], err_msg=x)
        assert out["free_head"].item() == ref["free_head"]


HARNESS = r"""
#include <pthread.h>
#include <stdint.h>
#include "swa_attn.h"
typedef swa_status (*plan_fn)(int, int, int, int, const int32_t*, const int32_t*, int32_t*, const int32_t*, int, const int32_t*, int,
                              int64_t*, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, void*, size_t, void*);
typedef struct {
  plan_fn f;
  int B, n, failed;
  void *lens, *table, *free_pages, *head, *slot, *pos, *row, *cu, *lens_out, *head_out, *stream;
} work;
static void* loop(void* x) {
  work* w = (work*)x;
  for (int i = 0; i < w->n; ++i)
    w->failed += w->f(w->B, 16, w->B, 2, w->lens, 0, w->table, w->free_pages, w->B, w->head, w->B, w->slot, w->pos, w->row, w->cu,
                      w->lens_out, w->head_out, 0, 0, w->stream) != SWA_OK;
  return 0;
}
void both(work* a, work* b) {
  pthread_t t, u;
  pthread_create(&t, 0, loop, a);
  pthread_create(&u, 0, loop, b);
  pthread_join(t, 0);
  pthread_join(u, 0);
}
"""


def test_plans_of_large_batches_from_two_threads(tmp_path):
    # both want more shared memory than a launch gets unasked, each its own
    # amount: neither takes away what the other has asked for
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    (tmp_path / "both.c").write_text(HARNESS)
    so = os.fspath(tmp_path / "both.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-pthread", "-I" + include, "-o", so, os.fspath(tmp_path / "both.c")], check=True)
    names = ("lens", "table", "free_pages", "head", "slot", "pos", "row", "cu", "lens_out", "head_out", "stream")

    class Work(ctypes.Structure):
        _fields_ = [("f", ctypes.c_void_p)] + [(x, ctypes.c_int) for x in ("B", "n", "failed")] + [(x, ctypes.c_void_p) for x in names]

    works, kept = [], []
    for B in (8192, 4300):
        zeros = lambda n, t=torch.int32: torch.zeros(n, dtype=t, device=dev())   # noqa: E731
        buf = [zeros(B), zeros(2 * B), torch.arange(B, dtype=torch.int32, device=dev()), zeros(1), zeros(B, torch.int64), zeros(B),
               zeros(B), zeros(B + 1), zeros(B), zeros(1)]
        stream = torch.cuda.Stream()
        kept.append((buf, stream))
        works.append(Work(ctypes.cast(swa.load("bf16").swa_kv4_plan, ctypes.c_void_p).value, B, 20000, 0,
                          *(t.data_ptr() for t in buf), stream.cuda_stream))
    torch.cuda.synchronize()
    ctypes.CDLL(so).both(ctypes.byref(works[0]), ctypes.byref(works[1]))
    torch.cuda.synchronize()
    assert [w.failed for w in works] == [0, 0]
    for (buf, _), w in zip(kept, works):
        assert torch.equal(buf[4].cpu(), 16 * torch.arange(w.B))


# ---------------------------------------------------------------------------
# Positions outside the tables
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("short_way", [False, True])
def test_rows_of_positions_outside_the_tables_are_zero_in_new_outputs(kind, inter, short_way, monkeypatch):
    swa.load(kind)
    if not short_way:
        monkeypatch.setattr(swa, "_fast", None)
    B, T, Hq, Hkv, d, rot = 2, 40, 5, 1, 128, 48
    q, k = randn(1, B, T, Hq, d, dtype=DT[kind]).to(dev()), randn(2, B, T, Hkv, d, dtype=DT[kind]).to(dev())
    rope = swa.rope_tables(30, rot)
    pos = torch.randint(0, 30, (B, T), generator=gen(3), dtype=torch.int32)
    bad = torch.rand(B, T, generator=gen(4)) < 0.3
    pos[bad] = torch.where(torch.rand(int(bad.sum()), generator=gen(5)) < 0.5, -1, 30).int()
    pd, bad = pos.to(dev()), bad.to(dev())
    qw, kw = swa.rope_apply(q, k, rope, pos=pd.clamp(0, 29), interleaved=inter)
    qw[bad], kw[bad] = 0, 0

    def stale():      # what the next allocations of these sizes find in memory
        a, b = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
        del a, b

    ws = torch.zeros(256, dtype=torch.uint8, device=dev())
    for w in (None, ws):
        stale()
        qo, ko = swa.rope_apply(q, k, rope, pos=pd, interleaved=inter, workspace=w)
        assert torch.equal(qo, qw) and torch.equal(ko, kw)
        stale()
        assert torch.equal(swa.rope_apply(None, k, rope, pos=pd, interleaved=inter, workspace=w)[1], kw)
        # an output of the caller's keeps those rows, a new one beside it is zero there
        mine = torch.full_like(q, 3.0)
        stale()
        qo, ko = swa.rope_apply(q, k, rope, pos=pd, interleaved=inter, out=(mine, None), workspace=w)
        assert qo is mine and torch.all(qo[bad] == 3.0) and torch.equal(qo[~bad], qw[~bad]) and torch.equal(ko, kw)
        same = k.clone()
        stale()
        qo, ko = swa.rope_apply(q, same, rope, pos=pd, interleaved=inter, out=(None, same), workspace=w)
        assert torch.equal(qo, qw) and torch.equal(ko[bad], k[bad]) and torch.equal(ko[~bad], kw[~bad])
    assert swa.swa_attn_check_status(ws) == swa.SWA_ERR_DEVICE_CHECK


# ---------------------------------------------------------------------------
# Rows whose squares pass fp32
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 48, True), (64, 0, False)])
@pytest.mark.parametrize("power,eps", [(100, 1e-6), (70, 0.0), (115, 1e-6)])
def test_keys_whose_squares_pass_fp32_are_normed(kind, d, rot, inter, power, eps):
    T, Hkv, page = 23, 3, 32
    k = randn(1, 1, T, Hkv, d, dtype=DT[kind])
    k[0, 1::2] *= 2.0 ** power               # beside rows of ordinary size
    tabs = None if not rot else tuple(torch.tensor(x, dtype=torch.float32) for x in dec.rope_tables(T, rot))
    gk = 1 + 0.1 * randn(3, d)
    cache = random_cache(9, 2, Hkv, page, d).to(dev())
    slot = torch.arange(T, device=dev()).view(1, T)
    swa.kv4_append(cache, k.to(dev()), randn(2, 1, T, Hkv, d, dtype=DT[kind]).to(dev()), slot, interleaved=inter, eps=eps,
                   rope=None if tabs is None else tuple(t.to(dev()) for t in tabs), gk=gk.to(dev()))
    kw = {} if tabs is None else dict(cos=f64(tabs[0])[:T], sin=f64(tabs[1])[:T], interleaved=inter)
    want, _, _, _ = dec.append_rows(f64(k)[0], f64(k)[0], f64(gk), float(np.float32(eps)), **kw)
    assert np.abs(want[1]).max() > 1         # normed, not vanished
    for t in range(T):
        sc = scales_of(cache.cpu(), page, t)
        nk, _ = numbers_of(cache.cpu(), page, t)
        check_held(want[t], nk, sc[0, :, :, 0], sc[0, :, :, 1], False, np.abs(want[t]).max(-1))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_an_infinite_key_entry_stays_in_its_group(kind):
    # x / inf = 0 beside it, inf / inf = NaN where it is
    d, page = 128, 16
    k = randn(1, 1, 4, 1, d, dtype=DT[kind])
    k[0, 1, 0, 5], k[0, 2, 0, 100] = math.inf, -math.inf
    cache = random_cache(1, 1, 1, page, d).to(dev())
    slot = torch.arange(4, device=dev()).view(1, 4)
    swa.kv4_append(cache, k.to(dev()), k.to(dev()), slot)
    kr = swa.kv4_read(cache, slot, dtype=torch.float32)[0][0, :, 0].cpu()
    assert torch.isnan(kr[1, :64]).all() and torch.all(kr[1, 64:] == 0)
    assert torch.isnan(kr[2, 64:]).all() and torch.all(kr[2, :64] == 0)
    assert torch.isfinite(kr[[0, 3]]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (64, 32, True), (64, 0, False)])
@pytest.mark.parametrize("power,eps", [(100, 1e-6), (70, 0.0), (115, 1e-6)])
def test_queries_whose_squares_pass_fp32_are_normed(kind, d, rot, inter, power, eps):
    lens, Hkv, page = [90, 5], 2, 32
    cache, table, rows = build_cache(lens, Hkv, d, page)
    q = randn(2, 2, 8, d, dtype=DT[kind])
    big = q.clone()
    big[:, 1::2] *= 2.0 ** power
    tabs = None if not rot else tuple(torch.tensor(x, dtype=torch.float32) for x in dec.rope_tables(90, rot))
    o, lse = swa.kv4_attention(cache.to(dev()), big.to(dev()), table.to(dev()), i32(*lens), interleaved=inter, eps=eps,
                               rope=None if tabs is None else tuple(t.to(dev()) for t in tabs))
    for b, n in enumerate(lens):
        kw = {} if tabs is None else dict(cos=f64(tabs[0])[n - 1], sin=f64(tabs[1])[n - 1], interleaved=inter)
        ro, rl = dec.attend(f64(big)[b], *rows[b], eps=float(np.float32(eps)), **kw)
        assert np.all(np.abs(f64(lse)[b] - rl) <= 1e-4)
        tol = HALF[kind] * np.abs(ro) + 1.7e-4 * np.abs(rows[b][1]).max()
        assert np.all(np.abs(f64(o)[b] - ro) <= tol)


# ---------------------------------------------------------------------------
# Tighter bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rot,rows,first,kw", [
    (128, 3000, 0, {}), (64, 500, 2 ** 20, {}), (16, 4000, 12345, {}), (128, 700, 1000, dict(base=500000.0)),
    (96, 700, 4000, dict(scaling="ntk", factor=8.0)), (64, 900, 65536, dict(scaling="by_parts", factor=16.0, orig_len=4096))])
def test_tables_keep_their_polynomials_error(rot, rows, first, kw):
    """With u = 2^-24 and |x| <= pi/4 the reduced angle: cutting the angle to 32
    bits costs 2 pi 2^-32 = 0.025 u; the integer's rounding, the constant's and
    the product's 3 u x, of which cosine sees 3 u x sin x <= 1.67 u and sine 3 u
    x cos x <= 1.67 u; Taylor's remainder x^10 / 10! = 2.5e-8 = 0.42 u (cosine),
    x^11 / 11! = 0.03 u (sine); x x rounded: y / 2 u = 0.31 u; the polynomial's
    last steps 0.5 u (the result lies within [1/2, 1]) + 0.2 u for the ones
    before. Sum 3.2 u. The oracle's own angle is off by its 2^-53 part."""
    cos, sin = swa.rope_tables(rows, rot, first=first, **kw)
    rc, rs = dec.rope_tables(rows, rot, first=first, **kw)
    tol = 3.2 * U + (first + rows) * 2.0 ** -52
    assert np.abs(f64(cos) - rc).max() <= tol
    assert np.abs(f64(sin) - rs).max() <= tol


def test_attention_in_fp32_keeps_the_third_term_of_p():
    """Two keys, logits so small (softmax_scale 2^-9) that their error does not
    count: the products of a logit sum to at most 0.15 in absolute value, so
    (see the attention's bound) it is off by 0.15 * 2.6e-6 = 4e-7, and by 2^-22
    through exp2 (2 ulp) = 2.4e-7; both enter o twice (numerator and sum). P
    times a step as three bf16 terms keeps 2^-24. The matrix instructions add
    three terms to sums that are rounded down to 2^-23 of them at most, four
    times; six fp32 roundings follow. Together 2 * 6.4e-7 + 4 * 2^-23 + 8 * 2^-24
    = 2.3e-6 of sum_j p_j (|s (n - 8)| + |z|) / sum_j p_j. Two terms alone would
    leave up to 2^-17 = 7.6e-6."""
    B, Hq, d, page = 64, 4, 64, 16
    cache, table, rows = build_cache([2] * B, 1, d, page)
    sc = cache[..., 16 * d:].view(torch.bfloat16).view(-1, 1, 1, 2, 16, 1, 2)
    for b in range(B):        # centres 0, numbers far from 8: the step's term is all there is
        pg = int(table[b, 0])
        sc[pg, 0, 0, 1, :2, 0, 1] = 0.0
        rows[b] = (rows[b][0], np.array([dec.read_row(cache.numpy()[pg:pg + 1], page, j, 0)[1] for j in range(2)])[:, None])
    q = randn(5, B, Hq, d)
    o, lse = swa.kv4_attention(cache.to(dev()), q.to(dev()), table.to(dev()), i32(*[2] * B), softmax_scale=2.0 ** -9)
    worst = 0.0
    for b in range(B):
        ro, rl = dec.attend(f64(q)[b], *rows[b], scale=2.0 ** -9)
        z = dec.rms_norm(f64(q)[b], None, EPS) @ rows[b][0][:, 0].T * 2.0 ** -9
        p = np.exp(z - z.max(-1, keepdims=True))
        weight = (p / p.sum(-1, keepdims=True)) @ np.abs(rows[b][1][:, 0])
        worst = max(worst, float((np.abs(f64(o)[b] - ro) / np.maximum(weight, 1e-30)).max()))
        assert np.abs(f64(lse)[b] - rl).max() <= 1e-6
    assert worst <= 2.5e-6, worst


# ---------------------------------------------------------------------------
# Block tables wider than the requests, and the largest batch
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,width,window", [(1, 8192, -1), (32, 4096, -1), (3, 8192, 700)])
def test_attention_with_a_table_much_wider_than_the_requests(B, width, window):
    # the parts of a request follow the table's width; its result is that of a
    # table of its own width to the rounding of the sums
    d, page, Hkv, Hq = 128, 16, 2, 8
    lens = [int(n) for n in np.random.default_rng(B).integers(1, 3000, B)]
    lens[0] = 3000
    held = [-(-n // page) for n in lens]
    cache = random_cache(1, sum(held), Hkv, page, d)
    sc = cache[..., 16 * d:].view(torch.bfloat16)
    sc[..., 0::2], sc[..., 1::2] = 0.2, (0.2 * randn(4, *sc[..., 1::2].shape)).bfloat16()
    ids, at = torch.randperm(sum(held), generator=gen(2)).int(), 0
    wide = torch.full((B, width), -1, dtype=torch.int32)
    for b in range(B):
        wide[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    cd, q = cache.to(dev()), randn(3, B, Hq, d).to(dev())
    ws = swa.new_kv4_workspace(cd, B, Hq, max_pages=width, window=window, kind="fp32")
    got = swa.kv4_attention(cd, q, wide.to(dev()), i32(*lens), window=window, workspace=ws)
    want = swa.kv4_attention(cd, q, wide[:, :max(held)].contiguous().to(dev()), i32(*lens), window=window, workspace=ws)
    assert swa.swa_attn_check_status(ws, kind="fp32") == swa.SWA_OK
    # the same logits bit for bit; exp2 over other maxima (2^-22) and sums of 3000
    # terms in another order, 24 roundings deep on either side, of nothing past 16
    for a, b in zip(got, want):
        assert (a - b).abs().max().item() <= 24 * 2 * U * 16
    slot = (wide[0].long().clamp(min=0)[:, None] * page + torch.arange(page)).view(1, -1)[:, :lens[0]].contiguous().to(dev())
    k, v = (x[0].double().cpu().numpy() for x in swa.kv4_read(cd, slot, dtype=torch.float32))
    ro, rl = dec.attend(f64(q)[0], k, v, window=window)
    assert np.abs(f64(got[1])[0] - rl).max() <= 1e-4
    assert np.all(np.abs(f64(got[0])[0] - ro) <= U * np.abs(ro) + 1.7e-4 * np.abs(v).max())


def test_attention_of_the_largest_batch():
    # 65535 rows of B, eight distinct ones repeated
    lens = [33, 1, 0, 64, 17, 90, 16, 5]
    cache, table, rows = build_cache(lens, 1, 64, 16)
    B = 65535
    at = torch.arange(B) % 8
    q = randn(2, 8, 1, 64, dtype=torch.bfloat16)
    cd = cache.to(dev())
    o, lse = swa.kv4_attention(cd, q[at].to(dev()), table[at].to(dev()), torch.tensor(lens, dtype=torch.int32)[at].to(dev()))
    small = swa.kv4_attention(cd, q.to(dev()), table.to(dev()), i32(*lens))
    for b in range(8):
        n = lens[b]
        if n:
            ro, rl = dec.attend(f64(q)[b], *rows[b])
            assert np.abs(f64(small[1])[b] - rl).max() <= 1e-4
            assert np.all(np.abs(f64(small[0])[b] - ro) <= 2.0 ** -8 * np.abs(ro) + 1.7e-4 * np.abs(rows[b][1]).max())
    at = at.to(dev())
    assert torch.equal(o, small[0][at]) and torch.equal(lse, small[1][at])
    with pytest.raises(swa.SwaError):
        swa.kv4_attention(cd, q[torch.zeros(65536, dtype=torch.long)].to(dev()), table[:1].expand(65536, -1).contiguous().to(dev()),
                          torch.ones(65536, dtype=torch.int32, device=dev()))

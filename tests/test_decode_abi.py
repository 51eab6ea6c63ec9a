"""Host-side checks of the rotary and decode entry points: sizes, and the
refusal of bad arguments before anything is launched. Nothing here runs on a
GPU; the addresses are never followed."""

import ctypes
import math

import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from sliding_window_gqa_qk_gb300 import build as swa_build

KINDS = ["bf16", "fp32"]
A = 1 << 20
BAD, UNS, WS = swa.SWA_ERR_INVALID_ARG, swa.SWA_ERR_UNSUPPORTED, swa.SWA_ERR_WORKSPACE
# What a call that passes every check ends with on a machine without a GPU.
PAST = (swa.SWA_ERR_CUDA, swa.SWA_ERR_UNSUPPORTED)

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses would be used")


@pytest.fixture(scope="session", autouse=True)
def built_libraries():
    swa_build.build()


def params(**kw):
    base = dict(B=2, T=3, Hq=4, Hkv=2, d=128)
    base.update(kw)
    return swa.make_params(**base)


def freq(**kw):
    base = dict(rot=64, scaling=swa.SWA_ROPE_PLAIN, base=1e4, factor=1.0, orig_len=0.0, slow=1.0, fast=32.0, amplitude=1.0)
    base.update(kw)
    return swa.swa_rope_freq(**base)


def rope(**kw):
    base = dict(cos=A, sin=A, rows=64, rot=64, interleaved=0)
    base.update(kw)
    return swa.swa_rope(**base)


def cache(**kw):
    base = dict(data=A, n_pages=10, page=32)
    base.update(kw)
    return swa.swa_kv4_cache(**base)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [
    dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=0), dict(rot=-16), dict(scaling=4), dict(scaling=-1), dict(base=0.5),
    dict(base=math.nan), dict(base=math.inf), dict(amplitude=-1.0), dict(amplitude=math.nan),
    dict(scaling=swa.SWA_ROPE_LINEAR, factor=0.5), dict(scaling=swa.SWA_ROPE_NTK, factor=math.nan),
    dict(scaling=swa.SWA_ROPE_BY_PARTS, factor=2.0), dict(scaling=swa.SWA_ROPE_BY_PARTS, factor=2.0, orig_len=100, slow=3, fast=3),
    dict(scaling=swa.SWA_ROPE_BY_PARTS, factor=2.0, orig_len=100, slow=-1.0),
])
def test_tables_refuse(kind, bad):
    assert swa.swa_rope_tables(freq(**bad), 0, 8, A, A, None, kind) == BAD


def test_tables_refuse_rows_and_addresses():
    for args in ((-1, 8, A, A), (0, -1, A, A), (0, 8, None, A), (0, 8, A, None), (0, 8, A + 8, A), (2 ** 31 - 4, 8, A, A)):
        assert swa.swa_rope_tables(freq(), *args) == BAD
    assert swa.load("bf16").swa_rope_tables(None, 0, 8, A, A, None) == BAD
    assert swa.swa_rope_tables(freq(), 5, 0, A, A) == swa.SWA_OK   # nothing to do


def apply(p, r, kind="bf16", **kw):
    a = dict(pos=None, q=A, k=A, q_out=A, k_out=A, inverse=0, ws=None, ws_bytes=0)
    a.update(kw)
    return swa.swa_rope_apply(p, r, a["pos"], a["q"], a["k"], a["q_out"], a["k_out"], a["inverse"], a["ws"],
                              a["ws_bytes"], None, kind)


@needs_no_gpu
@pytest.mark.parametrize("kind", KINDS)
def test_apply_refuses(kind):
    p = params()
    for r in (None, rope(cos=None), rope(sin=None), rope(cos=None, sin=None), rope(rot=8), rope(rot=40), rope(rot=144),
              rope(interleaved=2), rope(rows=0), rope(cos=A + 4)):
        assert apply(p, r, kind) == BAD
    assert apply(params(d=64), rope(rot=80), kind) == BAD          # past the head
    assert apply(p, rope(rows=2), kind) == BAD                     # T = 3 positions counted from 0
    assert apply(p, rope(rows=2), kind, pos=A) in PAST             # given ones are checked on the device
    for kw in (dict(inverse=2), dict(q_out=None), dict(k=None), dict(q=A + 8), dict(k_out=A + 2), dict(pos=A + 2),
               dict(ws=A + 16, ws_bytes=256)):
        assert apply(p, rope(), kind, **kw) == BAD
    assert apply(p, rope(), kind, ws=A, ws_bytes=255) == WS
    assert apply(params(d=96), rope(), kind) == UNS
    assert apply(params(Hq=3), rope(), kind) == BAD
    assert apply(params(B=0), rope(), kind) == swa.SWA_OK
    assert apply(p, rope(), kind, q=None, q_out=None, k=None, k_out=None) == swa.SWA_OK
    assert apply(p, rope(), kind) in PAST and apply(p, rope(), kind, k=None, k_out=None, ws=A, ws_bytes=256) in PAST


def test_cache_and_workspace_sizes():
    for d in (64, 128):
        p = params(d=d, Hq=6, Hkv=3, B=5, T=1)
        assert swa.swa_kv4_cache_size(p, 7, 48) == 7 * 3 * 3 * 18 * d
        for bad in ((0, 48), (7, 0), (7, 8), (7, 24), (7, 1 << 21), (-1, 16)):
            assert swa.swa_kv4_cache_size(p, *bad) == 0
        # past 32 bits
        assert swa.swa_kv4_cache_size(p, 1 << 24, 16) == (1 << 24) * 3 * 18 * d
        for kind in KINDS:
            n = swa.swa_kv4_workspace_size(p, 16, 4096, kind)
            assert n >= 256 and n % 256 == 0
            assert swa.swa_kv4_workspace_size(p, 24, 4096, kind) == 0
            assert swa.swa_kv4_workspace_size(p, 16, 0, kind) == 0
            assert swa.swa_kv4_workspace_size(p, 1 << 20, 1 << 12, kind) == 0
    assert swa.swa_kv4_cache_size(params(d=96), 7, 48) == 0
    assert swa.swa_kv4_workspace_init(None, 256) == BAD
    assert swa.swa_kv4_workspace_init(A + 1, 256) == BAD
    assert swa.swa_kv4_workspace_init(A, 256) == WS
    # the counters alone: what every call needs
    least = swa.swa_kv4_workspace_size(params(T=1, B=1, Hq=1, Hkv=1), 16, 1)
    assert swa.swa_kv4_workspace_init(A, least - 1) == WS


def plan(**kw):
    a = dict(n_pages=10, page=16, B=4, max_pages=8, lens=A, new=A, table=A, free=A, n_free=10, head=A, n_tokens=16, slot=A,
             pos=A, row=A, cu=A, lens_out=2 * A, head_out=2 * A, ws=None, ws_bytes=0)
    a.update(kw)
    return swa.swa_kv4_plan(a["n_pages"], a["page"], a["B"], a["max_pages"], a["lens"], a["new"], a["table"], a["free"],
                            a["n_free"], a["head"], a["n_tokens"], a["slot"], a["pos"], a["row"], a["cu"], a["lens_out"],
                            a["head_out"], a["ws"], a["ws_bytes"])


@needs_no_gpu
def test_plan_refuses():
    for kw in (dict(page=8), dict(page=0), dict(n_pages=0), dict(B=-1), dict(max_pages=0), dict(n_free=-1), dict(n_tokens=-1),
               dict(max_pages=1 << 27), dict(max_pages=(1 << 27) - 4), dict(n_tokens=2 ** 31 - 1), dict(lens=None), dict(table=None), dict(free=None),
               dict(head=None), dict(slot=None), dict(pos=None), dict(row=None), dict(cu=None), dict(lens_out=None),
               dict(head_out=None), dict(slot=A + 8), dict(pos=A + 4), dict(row=A + 4), dict(lens=A + 2),
               dict(lens_out=A), dict(lens=3 * A, lens_out=A), dict(head_out=A), dict(ws=A + 8, ws_bytes=256)):
        assert plan(**kw) == BAD, kw
    assert plan(B=8193) == UNS
    assert plan(ws=A, ws_bytes=8) == WS
    assert plan() in PAST and plan(new=None) in PAST and plan(ws=A, ws_bytes=256) in PAST


def append(p, c, r=None, ex=None, kind="bf16", **kw):
    a = dict(k=A, v=A, gk=None, ve=None, tok=None, gate=None, pos=None, slot=A, ws=None, ws_bytes=0)
    a.update(kw)
    return swa.swa_kv4_append(p, ex, c, r, a["k"], a["v"], a["gk"], a["ve"], a["tok"], a["gate"], a["pos"], a["slot"],
                              a["ws"], a["ws_bytes"], None, kind)


def read(p, c, kind="bf16", **kw):
    a = dict(slot=A, k=A, v=A, ws=None, ws_bytes=0)
    a.update(kw)
    return swa.swa_kv4_read(p, c, a["slot"], a["k"], a["v"], a["ws"], a["ws_bytes"], None, kind)


def attn(p, c, r=None, ex=None, kind="bf16", **kw):
    a = dict(q=A, gq=None, table=A, max_pages=16, lens=A, o=A, lse=A, ws=A, ws_bytes=1 << 40)
    a.update(kw)
    return swa.swa_kv4_attn(p, ex, c, r, a["q"], a["gq"], a["table"], a["max_pages"], a["lens"], a["o"], a["lse"], a["ws"],
                            a["ws_bytes"], None, kind)


@needs_no_gpu
@pytest.mark.parametrize("kind", KINDS)
def test_cache_calls_refuse(kind):
    p, one = params(), params(T=1)
    for c in (None, cache(data=None), cache(data=A + 8), cache(n_pages=0), cache(page=0), cache(page=24)):
        assert append(p, c, kind=kind) == BAD
        assert read(p, c, kind) == BAD
        assert attn(one, c, kind=kind) == BAD
    assert append(p, cache(page=1 << 21), kind=kind) == UNS
    assert append(params(d=96), cache(), kind=kind) == UNS and attn(params(d=96, T=1), cache(), kind=kind) == UNS
    for kw in (dict(k=None), dict(v=None), dict(slot=None), dict(k=A + 8), dict(v=A + 4), dict(slot=A + 4), dict(pos=A + 1),
               dict(gk=A + 2), dict(tok=A + 2), dict(gate=A + 1), dict(ws=A + 1, ws_bytes=256)):
        assert append(p, cache(), kind=kind, **kw) == BAD, kw
    assert append(p, cache(), kind=kind, ws=A, ws_bytes=128) == WS
    assert append(p, cache(), rope(rows=2), kind=kind) == BAD
    assert append(p, cache(), rope(rows=2), kind=kind, pos=A) in PAST
    assert append(p, cache(), rope(rot=72), kind=kind) == BAD
    ex = swa.swa_extras(rope_cos=A, rope_sin=A, rope_rows=64)
    assert append(p, cache(), ex=ex, kind=kind) == BAD               # rotary comes as swa_rope here
    assert attn(one, cache(), ex=ex, kind=kind) == BAD
    pv = params(vocab=7)
    assert append(pv, cache(), kind=kind, ve=A) == BAD               # no token ids
    assert append(p, cache(), kind=kind, ve=A, tok=A) == BAD         # vocab 0
    assert append(pv, cache(), kind=kind, ve=A + 8, tok=A) == BAD
    gate = swa.swa_extras(gate_x=A, gate_x_stride=32, gate_w=A, gate_ch=33)
    assert append(pv, cache(), ex=gate, kind=kind, ve=A, tok=A) == BAD
    gate = swa.swa_extras(gate_x=A, gate_x_stride=32, gate_w=A, gate_ch=32)
    assert append(pv, cache(), ex=gate, kind=kind, ve=A, tok=A, gate=A) == BAD   # two gates
    assert append(pv, cache(), ex=gate, kind=kind, ve=A, tok=A) in PAST
    assert append(params(B=0), cache(), kind=kind) == swa.SWA_OK and read(params(T=0), cache(), kind) == swa.SWA_OK
    assert append(p, cache(), rope(), kind=kind) in PAST and read(p, cache(), kind) in PAST
    for kw in (dict(slot=None), dict(k=None), dict(v=A + 8), dict(slot=A + 4), dict(ws=A + 2, ws_bytes=256)):
        assert read(p, cache(), kind, **kw) == BAD, kw
    for kw in (dict(q=None), dict(table=None), dict(lens=None), dict(o=None), dict(lse=None), dict(q=A + 8), dict(lens=A + 2),
               dict(gq=A + 8), dict(lse=A + 2), dict(table=A + 1), dict(max_pages=0), dict(max_pages=1 << 27), dict(max_pages=(1 << 26) - 2), dict(ws=None), dict(ws=A + 16)):
        assert attn(one, cache(), kind=kind, **kw) == BAD, kw
    assert attn(one, cache(), kind=kind, ws_bytes=swa.swa_kv4_workspace_size(one, 32, 16, kind) - 1) == WS
    assert attn(params(T=2), cache(), kind=kind) == BAD and attn(params(T=1, causal=False), cache(), kind=kind) == BAD
    assert attn(params(T=1, window=-2), cache(), kind=kind) == BAD
    assert attn(params(T=1, B=0), cache(), kind=kind) == swa.SWA_OK
    assert attn(one, cache(), rope(rows=2), kind=kind) in PAST and attn(one, cache(), kind=kind) in PAST


def test_convenience_calls_refuse_types_and_shapes():
    c = torch.zeros(4, 2, 2, 18 * 64, dtype=torch.uint8)
    k = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16)
    slot, lens = torch.zeros(1, 3, dtype=torch.int64), torch.ones(1, dtype=torch.int32)
    table, q = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    calls = [
        lambda: swa.kv4_append(c.float(), k, k, slot), lambda: swa.kv4_append(c[:, :, :, :100], k, k, slot),
        lambda: swa.kv4_append(c, k.half(), k.half(), slot), lambda: swa.kv4_append(c, k, k.float(), slot),
        lambda: swa.kv4_append(c, k, k[:, :2], slot), lambda: swa.kv4_append(c, k, k, slot.int()),
        lambda: swa.kv4_append(c, k, k, slot, pos=slot), lambda: swa.kv4_append(c, k, k, slot[:, :2]),
        lambda: swa.kv4_append(c, k.transpose(1, 2), k, slot),
        lambda: swa.kv4_append(c, k, k, slot, rope=(torch.zeros(4, 32, dtype=torch.float64),) * 2),
        lambda: swa.kv4_append(c, k, k, slot, gk=torch.ones(32)),
        lambda: swa.kv4_append(c, k, k, slot, ve=torch.zeros(9, 64, dtype=torch.bfloat16), tok=lens),
        lambda: swa.kv4_read(c, slot.int()), lambda: swa.kv4_read(c, slot[0]),
        lambda: swa.kv4_attention(c, q, table.long(), lens), lambda: swa.kv4_attention(c, q, table, lens.long()),
        lambda: swa.kv4_attention(c, q[..., :32], table, lens), lambda: swa.kv4_attention(c, q.half(), table, lens),
        lambda: swa.kv4_attention(c, q, table[0], lens), lambda: swa.kv4_attention(c, q, table, torch.ones(2, dtype=torch.int32)),
        lambda: swa.kv4_plan(lens.long(), None, table, lens, lens, page=16, n_pages=4),
        lambda: swa.kv4_plan(lens, lens, table, lens, lens, page=16, n_pages=4),
        lambda: swa.kv4_plan(lens, None, table[0], lens, lens, page=16, n_pages=4),
        lambda: swa.rope_apply(None, None, None), lambda: swa.rope_apply(k.half(), None, None),
        lambda: swa.rope_apply(k, k[:, :2], None), lambda: swa.rope_tables(8, 16, scaling="other", device="cpu"),
        # right in every other way, but not on a GPU
        lambda: swa.kv4_append(c, k, k, slot), lambda: swa.kv4_read(c, slot), lambda: swa.kv4_attention(c, q, table, lens),
        lambda: swa.kv4_plan(lens, None, table, lens, lens, page=16, n_pages=4),
        lambda: swa.rope_tables(8, 16, device="cpu"), lambda: swa.rope_apply(k, None, (torch.zeros(4, 32),) * 2),
    ]
    for i, f in enumerate(calls):
        with pytest.raises(ValueError):
            f()
            print("call", i, "was taken")
    with pytest.raises(swa.SwaError):
        swa.new_kv4_cache(4, 24, 2, 64, "cpu")
    with pytest.raises(swa.SwaError):
        swa.new_kv4_cache(4, 16, 2, 96, "cpu")

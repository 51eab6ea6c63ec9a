"""Host-side checks of the norm, the 4-bit projections and the drafted tokens'
entry points: sizes, and the refusal of bad arguments before anything is
launched. Nothing here runs on a GPU; the addresses are never followed."""

import math

import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from sliding_window_gqa_qk_gb300 import build as swa_build

KINDS = ["bf16", "fp32"]
A, X = 1 << 20, 1 << 21
BAD, UNS, WS, OK = swa.SWA_ERR_INVALID_ARG, swa.SWA_ERR_UNSUPPORTED, swa.SWA_ERR_WORKSPACE, swa.SWA_OK
# What a call that passes every check ends with on a machine without a GPU.
PAST = (swa.SWA_ERR_CUDA, swa.SWA_ERR_UNSUPPORTED)
needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses would be used")


@pytest.fixture(scope="session", autouse=True)
def built_libraries():
    swa_build.build()


def norm(kind="bf16", **kw):
    a = dict(rows=4, C=64, eps=1e-6, x=A, add=None, gain=None, h=None, y=X, y8=None, scale=None, rstd=None)
    a.update(kw)
    return swa.swa_rms_norm(*a.values(), None, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(C=0), dict(C=4), dict(C=60), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(x=None),
    dict(y=None), dict(y8=X, scale=A), dict(y=None, y8=X), dict(scale=A), dict(add=A), dict(h=X), dict(x=A + 8), dict(y=X + 4),
    dict(gain=A + 4), dict(add=A + 8, h=A), dict(rstd=A + 2), dict(y=None, y8=X, scale=A + 1), dict(add=A, h=A + 8),
])
def test_norm_refuses(kind, bad):
    assert norm(kind, **bad) == BAD


def test_norm_limits():
    assert norm(C=65544) == UNS and norm(rows=2 ** 31) == UNS
    assert norm(rows=0, x=None) == OK
    assert swa.swa_rms_norm_workspace_size(10, 60) == 0 and swa.swa_rms_norm_workspace_size(-1, 64) == 0
    for rows in (0, 1, 7, 8, 9, 100, 10 ** 6):
        for C in (8, 768, 1024, 1032, 4096, 8192, 16384, 65536):
            for kind in KINDS:
                assert swa.swa_rms_norm_workspace_size(rows, C, kind) >= 4 * C


def back(kind="bf16", **kw):
    a = dict(rows=4, C=64, h=A, rstd=A, gain=None, dy=A, dh=None, dx=X, dgain=X, ws=A, n=1 << 20)
    a.update(kw)
    return swa.swa_rms_norm_bwd(*a.values(), None, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(C=12), dict(h=None), dict(rstd=None), dict(dy=None), dict(dx=None), dict(ws=None), dict(ws=A + 16),
    dict(h=A + 8), dict(dy=A + 8), dict(dh=A + 8), dict(dx=A + 8), dict(gain=A + 4), dict(dgain=A + 2), dict(rstd=A + 1),
])
def test_norm_backward_refuses(kind, bad):
    assert back(kind, **bad) == BAD


def test_norm_backward_workspace():
    n = swa.swa_rms_norm_workspace_size(4, 64)
    assert back(n=n - 1) == WS and back(rows=4, C=65544) == UNS


def lin(kind="bf16", **kw):
    a = dict(M=3, N=40, K=72, x=A, x_scale=None, w4=A, add=None, y=X)
    a.update(kw)
    return swa.swa_w4_linear(*a.values(), None, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(N=-3), dict(K=0), dict(K=4), dict(K=70), dict(x=None), dict(w4=None), dict(y=None), dict(x=A + 8),
    dict(w4=A + 8), dict(y=X + 8), dict(add=A + 8), dict(x_scale=A + 2), dict(y=A),
])
def test_linear_refuses(kind, bad):
    assert lin(kind, **bad) == BAD


def test_w4_sizes_and_limits():
    assert swa.swa_w4_size(16, 64) == 544 and swa.swa_w4_size(17, 72) == 4 * 544 and swa.swa_w4_size(1, 8) == 544
    assert swa.swa_w4_size(1 << 24, 1 << 24) == (1 << 20) * (1 << 18) * 544
    for N, K in ((0, 64), (16, 0), (16, 60), (-1, 64), ((1 << 24) + 1, 64), (16, (1 << 24) + 8)):
        assert swa.swa_w4_size(N, K) == 0
    assert lin(N=(1 << 24) + 1) == UNS and lin(M=0, x=None) == OK
    for f in (swa.swa_w4_pack, swa.swa_w4_unpack):
        assert f(0, 64, A, A, None, "bf16") == BAD and f(16, 64, None, A, None, "bf16") == BAD
        assert f(16, 64, A, None, None, "bf16") == BAD and f(16, 64, A + 8, A, None, "bf16") == BAD


def tree(**kw):
    a = dict(B=2, n=10, max_new=8, parent=A, cu=A, lens=A, pos=X, seen=X, ws=None, nws=None)
    a.update(kw)
    return swa.swa_kv4_tree(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(n=-1), dict(max_new=0), dict(max_new=-1), dict(B=0), dict(parent=None), dict(cu=None), dict(lens=None),
    dict(pos=None), dict(seen=None), dict(parent=A + 1), dict(seen=X + 4), dict(pos=X + 2), dict(ws=A + 16, nws=256),
])
def test_tree_refuses(bad):
    assert tree(**bad) == BAD


def test_tree_limits():
    assert tree(max_new=65) == UNS and tree(ws=A, nws=255) == WS and tree(n=0, parent=None) == OK and tree(B=0, n=0) == OK


def params(**kw):
    a = dict(B=2, T=1, Hq=4, Hkv=2, d=128)
    a.update(kw)
    return swa.make_params(**a)


def cache(**kw):
    a = dict(data=A, n_pages=10, page=32)
    a.update(kw)
    return swa.swa_kv4_cache(**a)


def attn(kind="bf16", p=None, ex=None, c=None, r=None, **kw):
    a = dict(n=10, max_new=8, q=A, gq=None, table=A, max_pages=4, lens=A, cu=A, pos=A, seen=A, o=X, lse=X, ws=A, nws=1 << 24)
    a.update(kw)
    return swa.swa_kv4_tree_attn(params() if p is None else p, ex, cache() if c is None else c, r, *a.values(), None, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [
    dict(p=params(T=2)), dict(p=params(causal=0)), dict(p=params(Hq=3)), dict(p=params(window=-2)), dict(n=-1), dict(max_new=0),
    dict(q=None), dict(table=None), dict(lens=None), dict(cu=None), dict(pos=None), dict(seen=None), dict(o=None), dict(lse=None),
    dict(q=A + 8), dict(o=X + 8), dict(gq=A + 4), dict(seen=A + 4), dict(pos=A + 1), dict(cu=A + 2), dict(ws=None), dict(ws=A + 64),
    dict(max_pages=0), dict(max_pages=1 << 27), dict(c=cache(page=24)), dict(c=cache(data=None)), dict(c=cache(data=A + 8)),
    dict(p=params(B=0)), dict(r=swa.swa_rope(A, None, 64, 64, 0)), dict(r=swa.swa_rope(A, A, 64, 24, 0)),
])
def test_tree_attention_refuses(kind, bad):
    assert attn(kind, **bad) == BAD


def test_tree_attention_limits():
    assert attn(p=params(d=96)) == UNS and attn(max_new=65) == UNS
    assert attn(nws=swa.swa_kv4_workspace_size(params(), 32, 4) - 1) == WS
    assert attn(n=0, q=None) == OK and attn(p=params(B=0), n=0) == OK
    assert attn(p=params(B=2048, Hq=64, Hkv=1), max_new=64) == UNS        # B * Hq


def move(p=None, c=None, **kw):
    a = dict(src=A, dst=X, ws=None, nws=None)
    a.update(kw)
    return swa.swa_kv4_move(params(T=5) if p is None else p, cache() if c is None else c, *a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(src=None), dict(dst=None), dict(src=A + 4), dict(dst=X + 4), dict(c=cache(n_pages=0)), dict(c=cache(page=8)),
    dict(c=cache(data=None)), dict(p=params(T=-1)), dict(p=params(B=-1)), dict(ws=A + 8, nws=256),
])
def test_move_refuses(bad):
    assert move(**bad) == BAD


def test_move_limits():
    assert move(p=params(T=65)) == UNS and move(p=params(B=0, T=5), src=None) == OK and move(p=params(T=0)) == OK
    assert move(ws=A, nws=128) == WS


@needs_no_gpu
def test_calls_that_pass_every_check_end_at_the_device():
    for kind in KINDS:
        assert norm(kind) in PAST and back(kind) in PAST and lin(kind) in PAST and attn(kind) in PAST
    assert attn(p=params(B=2047, Hq=32, Hkv=1), max_new=64, n=2047) in PAST
    assert tree() in PAST and move() in PAST and norm(y=None, y8=X, scale=A) in PAST and lin(x_scale=A) in PAST


# ---------------------------------------------------------------------------
# The Python functions tell what is wrong before anything is launched.
# ---------------------------------------------------------------------------

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


F32, I32, I64, U8, F8 = torch.float32, torch.int32, torch.int64, torch.uint8, torch.float8_e4m3fn


@pytest.mark.parametrize("call", [
    lambda: swa.rms_norm(t(2, 64, dtype=torch.float16)),
    lambda: swa.rms_norm(t(2, 64), t(64)),
    lambda: swa.rms_norm(t(2, 64), t(32, dtype=F32)),
    lambda: swa.rms_norm(t(2, 64), add=t(2, 64, dtype=F32)),
    lambda: swa.rms_norm(t(64, 2).T),
    lambda: swa.rms_norm(torch.zeros((), dtype=F32)),
    lambda: swa.rms_norm(t(2, 64)),                                               # not on a GPU
    lambda: swa.rms_norm_backward(t(2, 64), t(2), t(2, 64)),
    lambda: swa.rms_norm_backward(t(2, 64), t(2, dtype=F32), t(2, 64, dtype=F32)),
    lambda: swa.rms_norm_backward(t(2, 64), t(3, dtype=F32), t(2, 64)),
    lambda: swa.w4_pack(t(4, 64, dtype=I32)),
    lambda: swa.w4_pack(t(64)),
    lambda: swa.w4_unpack(t(1, 1, 544, dtype=U8), 17, 64),
    lambda: swa.w4_linear(t(2, 64), t(1, 2, 544, dtype=U8)),
    lambda: swa.w4_linear(t(2, 64), t(1, 1, 544, dtype=U8), out_features=17),
    lambda: swa.w4_linear(t(2, 64), t(1, 544, dtype=U8)),
    lambda: swa.w4_linear(t(2, 64), t(1, 1, 544, dtype=U8), dtype=F32),
    lambda: swa.w4_linear(t(2, 64, dtype=F8), t(1, 1, 544, dtype=U8)),
    lambda: swa.w4_linear(t(2, 64), t(1, 1, 544, dtype=U8), scale=t(2, dtype=F32)),
    lambda: swa.w4_linear(t(2, 64), t(1, 1, 544, dtype=U8), add=t(2, 15)),
    lambda: swa.kv4_tree(t(4, dtype=I64), t(2, dtype=I32), t(1, dtype=I32), max_new=4),
    lambda: swa.kv4_tree(t(4, dtype=I32), t(2, dtype=I32), t(2, dtype=I32), max_new=4),
    lambda: swa.kv4_move(t(1, 1, 1, 1152, dtype=U8), t(4, dtype=I64), t(4, dtype=I64)),
    lambda: swa.kv4_move(t(1, 1, 1, 1152, dtype=U8), t(1, 4, dtype=I64), t(1, 4, dtype=I32)),
    lambda: swa.kv4_tree_attention(t(1, 1, 1, 1152, dtype=U8), t(4, 2, 128), t(1, 1, dtype=I32), t(1, dtype=I32), t(2, dtype=I32),
                                   t(4, dtype=I32), t(4, dtype=I64), max_new=4),   # another head dim
    lambda: swa.kv4_tree_attention(t(1, 1, 1, 1152, dtype=U8), t(4, 2, 64), t(1, 1, dtype=I32), t(1, dtype=I32), t(3, dtype=I32),
                                   t(4, dtype=I32), t(4, dtype=I64), max_new=4),
])
def test_python_refuses(call):
    with pytest.raises(ValueError):
        call()


def block(kind="bf16", p=None, ex=None, c=None, r=None, w=None, **kw):
    a = dict(n=10, max_new=8, x=A, add=None, gain=None, gq=None, gk=None, ve=None, tok=None, slot=A, pos=A, cu=A, seen=A, table=A,
             max_pages=4, lens=A, out=X, ws=A, nws=1 << 28)
    a.update(kw)
    w = swa.swa_kv4_weights(64, A, A, A, A) if w is None else w
    return swa.swa_kv4_block(params() if p is None else p, ex, cache() if c is None else c, r, w, *a.values(), None, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [
    dict(p=params(T=2)), dict(p=params(causal=0)), dict(p=params(Hq=3)), dict(w=swa.swa_kv4_weights(60, A, A, A, A)),
    dict(w=swa.swa_kv4_weights(64, A, None, A, A)), dict(w=swa.swa_kv4_weights(64, A, A, A, A + 8)), dict(n=-1), dict(cu=None),
    dict(seen=None), dict(cu=None, seen=None), dict(x=None), dict(out=None), dict(out=A), dict(add=X), dict(slot=None), dict(pos=None),
    dict(table=None), dict(lens=None), dict(max_pages=0), dict(ws=None), dict(ws=A + 64), dict(gain=A + 4), dict(gq=A + 8),
    dict(slot=A + 4), dict(seen=A + 4), dict(ve=A), dict(ve=A, tok=A), dict(max_new=0), dict(c=cache(page=8)), dict(c=cache(data=None)),
    dict(r=swa.swa_rope(A, A, 0, 64, 0)), dict(ex=swa.swa_extras(gate_w=A, gate_ch=65)), dict(ex=swa.swa_extras(gate_w=A, gate_ch=33)),
    dict(ex=swa.swa_extras(gate_x=A)), dict(ex=swa.swa_extras(rope_cos=A)),
])
def test_block_refuses(kind, bad):
    assert block(kind, **bad) == BAD


def test_block_limits():
    n = swa.swa_kv4_block_workspace_size(params(), 64, 10)
    assert n > swa.swa_kv4_workspace_size(params(), 32, 4)
    assert block(nws=n - 1) == WS and block(n=0, x=None, nws=1 << 28) == OK and block(max_new=65) == UNS
    assert block(w=swa.swa_kv4_weights(65544, A, A, A, A)) == UNS
    assert swa.swa_kv4_block_workspace_size(params(T=2), 64, 10) == 0 and swa.swa_kv4_block_workspace_size(params(), 60, 10) == 0
    if not torch.cuda.is_available():
        assert block() in PAST and block(n=2, cu=None, seen=None) in PAST

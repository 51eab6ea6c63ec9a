"""Refusals and limits of the serving calls beside those of test_serve_abi.py.
Nothing here runs on a GPU; the addresses are never followed."""

import ctypes

import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from test_serve_abi import A, BAD, KINDS, X, attn, back, block, built_libraries, lin, move, norm, params, tree  # noqa: F401  (a fixture)


@pytest.mark.parametrize("kind", KINDS)
def test_norm_refuses_8_bit_rows_over_what_it_reads(kind):
    # (numbers of 8 bits over rows of 16 or 32: those of one row lie over entries of others, which are read by then or not)
    add = X + (1 << 20)
    for bad in (dict(x=A, y8=A), dict(x=A, add=add, h=X, y8=add), dict(x=A, add=add, h=A, y8=A), dict(x=A, add=add, h=X, y8=X)):
        assert norm(kind, y=None, scale=A, **bad) == BAD
        assert norm(kind, y=None, scale=A, rows=0, **bad) == swa.SWA_OK


def test_rows_of_a_projection_have_a_limit():
    # tiles of up to 256 rows, counted in 31 bits
    for kind in KINDS:
        for M in (2 ** 31 - 1, 2 ** 31 - 255):
            assert lin(kind, M=M) == swa.SWA_ERR_UNSUPPORTED and lin(kind, M=M, x_scale=A) == swa.SWA_ERR_UNSUPPORTED
            assert block(kind, n=M, nws=1 << 62) == swa.SWA_ERR_UNSUPPORTED
            assert swa.swa_kv4_block_workspace_size(params(), 64, M, kind) == 0
        if not torch.cuda.is_available():
            assert lin(kind, M=2 ** 31 - 256) == swa.SWA_ERR_CUDA
        assert swa.swa_kv4_block_workspace_size(params(), 64, 2 ** 31 - 256, kind) > 2 ** 38


FAR = [2 ** 31, 2 ** 32 + 5, 2 ** 40, -2 ** 31 - 1, -2 ** 40]


@pytest.mark.parametrize("n", FAR)
def test_numbers_that_do_not_fit_32_bits_are_refused(n):
    # (ctypes cuts them: a window of 2^40 became one of 0 keys)
    for call in (lambda: swa.make_params(1, 1, 2, 1, 128, window=n), lambda: swa.make_params(n, 1, 2, 1, 128),
                 lambda: swa.make_params(1, 1, 2, 1, 128, vocab=n), lambda: swa.swa_params(window=n), lambda: swa.swa_rope(A, A, n, 64, 0),
                 lambda: swa.swa_kv4_cache(A, n, 32), lambda: swa.swa_kv4_cache(A, 10, page=n), lambda: swa.swa_kv4_weights(n, A, A, A, A),
                 lambda: swa.swa_block_weights(n, A, A, A, A), lambda: swa.swa_rope_freq(rot=n)):
        with pytest.raises(ValueError):
            call()
    m = n + 64 if n > 0 else n - 64       # cut, some would be sizes that there are
    for call in (lambda: swa.swa_w4_size(m, 64), lambda: swa.swa_kv4_tree(2, 10, m, A, A, A, X, X),
                 lambda: swa.swa_w4_pack(m, 64, A, X, None, "bf16"), lambda: lin(M=m), lambda: norm(C=m),
                 lambda: swa.swa_kv4_block_workspace_size(params(), m, 10)):
        with pytest.raises((ValueError, ctypes.ArgumentError)):
            call()
    assert swa.make_params(1, 1, 2, 1, 128, window=2 ** 31 - 1).window == 2 ** 31 - 1
    e = swa.make_extras(wait_limit_ns=2 ** 40)
    assert e.wait_limit_ns == 2 ** 40


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses would be used")
@pytest.mark.parametrize("kind", KINDS)
def test_calls_that_pass_every_check_end_at_the_device_and_nowhere_else(kind):
    # asking for a device fails here; a check that refused a legal call as unsupported would answer otherwise
    end = swa.SWA_ERR_CUDA
    for bad in (dict(), dict(y=None, y8=X, scale=A), dict(C=65536), dict(rows=2 ** 31 - 1), dict(C=8), dict(y=A), dict(add=X, h=A, y=X)):
        assert norm(kind, **bad) == end
    for bad in (dict(), dict(dgain=None, ws=None), dict(dx=A), dict(C=65536, n=1 << 40)):
        assert back(kind, **bad) == end
    for bad in (dict(), dict(x_scale=A), dict(add=X), dict(M=1, N=1, K=8), dict(M=2 ** 31 - 256), dict(N=1 << 24, K=1 << 24)):
        assert lin(kind, **bad) == end
    assert swa.swa_w4_pack(1 << 24, 8, A, X, None, kind) == end and swa.swa_w4_unpack(16, 1 << 24, A, X, None, kind) == end
    assert tree() == end and tree(max_new=64, B=1) == end and tree(ws=A, nws=256) == end
    assert move() == end and move(p=params(T=64)) == end and move(ws=A, nws=256) == end
    for bad in (dict(), dict(max_new=64), dict(p=params(Hq=32, B=2047, Hkv=1), max_new=64, n=2047), dict(p=params(window=0)),
                dict(p=params(d=64)), dict(r=swa.swa_rope(A, A, 64, 64, 0)), dict(p=params(B=65535, Hq=1, Hkv=1), n=65535, max_new=1)):
        assert attn(kind, **bad) == end
    for bad in (dict(), dict(n=2, cu=None, seen=None), dict(add=A + 4096), dict(ve=A, tok=A, p=params(vocab=3)), dict(max_new=64),
                dict(ex=swa.swa_extras(wait_limit_ns=1)), dict(ex=swa.swa_extras(gate_w=A, gate_ch=32))):
        assert block(kind, **bad) == end


def test_what_a_weight_loses_as_bf16():
    # s (n - 8) for every step of one binade, as the calls of more than 32 rows round it: below 2^-8 of it (half a step of
    # 8 bits), and for some more than 2^-9. In sums that cancel, 2^-8 of the sum of sizes can exceed y's own rounding.
    s = (torch.arange(128, 256).float() / 128).view(-1, 1)
    assert torch.equal(s, s.bfloat16().float())
    exact = s.double() * torch.arange(1, 9).double()
    lost = ((exact.bfloat16().double() - exact).abs() / exact).max().item()
    assert 2.0 ** -9 < lost < 2.0 ** -8

"""Refusals and limits of the serving calls beside those of test_serve_abi.py.
Nothing here runs on a GPU; the addresses are never followed."""

import ctypes

import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from test_serve_abi import A, BAD, KINDS, X, block, built_libraries, lin, norm, params  # noqa: F401  (a fixture)


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

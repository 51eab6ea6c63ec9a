"""Refusals and limits of the serving calls beside those of test_serve_abi.py.
Nothing here runs on a GPU; the addresses are never followed."""

import pytest

import sliding_window_gqa_qk_gb300 as swa
from test_serve_abi import A, BAD, KINDS, X, built_libraries, norm  # noqa: F401  (a fixture)


@pytest.mark.parametrize("kind", KINDS)
def test_norm_refuses_8_bit_rows_over_what_it_reads(kind):
    # (numbers of 8 bits over rows of 16 or 32: those of one row lie over entries of others, which are read by then or not)
    add = X + (1 << 20)
    for bad in (dict(x=A, y8=A), dict(x=A, add=add, h=X, y8=add), dict(x=A, add=add, h=A, y8=A), dict(x=A, add=add, h=X, y8=X)):
        assert norm(kind, y=None, scale=A, **bad) == BAD
        assert norm(kind, y=None, scale=A, rows=0, **bad) == swa.SWA_OK

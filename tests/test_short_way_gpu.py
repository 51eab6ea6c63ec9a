"""The binding's short way into the rotary and decode calls (csrc/py_fast.cpp),
with functions bound in place of the library's: a call is made once, its errors
are told, and other Python threads run beside it. No call here fails on the GPU."""

import ctypes
import os
import subprocess
import threading
import time

import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from test_decode_gpu import dev, randn

pytestmark = pytest.mark.gpu

NAMES = ("swa_rope_tables", "swa_rope_apply", "swa_kv4_plan", "swa_kv4_append", "swa_kv4_read", "swa_kv4_attn")


@pytest.fixture
def bind():
    """bind(name, function): the bf16 library's entry point of that name, as
    the short way sees it, for the time of a test."""
    lib = swa.load("bf16")
    assert swa._fast is not None, "the short way is not built"
    real = {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in NAMES}
    kept = []

    def put(name, f):
        g = f if not callable(f) or isinstance(f, ctypes._CFuncPtr) else ctypes.CFUNCTYPE(ctypes.c_int, *getattr(lib, name).argtypes)(f)
        kept.append(g)
        assert swa._fast.bind(0, *(ctypes.cast(g, ctypes.c_void_p).value if n == name else real[n] for n in NAMES))

    yield put
    assert swa._fast.bind(0, *real.values())


def calls():
    """One ordinary call of each entry point, as functions."""
    i32 = dict(dtype=torch.int32, device=dev())
    cache = swa.new_kv4_cache(4, 16, 2, 64, dev())
    ws = swa.new_kv4_workspace(cache, 1, 4, max_pages=4)
    k, q = randn(1, 1, 3, 2, 64, dtype=torch.bfloat16).to(dev()), randn(2, 1, 4, 64, dtype=torch.bfloat16).to(dev())
    slot = torch.arange(3, device=dev()).view(1, 3)
    table, lens, rope = torch.zeros(1, 4, **i32), torch.full((1,), 3, **i32), swa.rope_tables(8, 64)
    return {
        "swa_rope_tables": lambda: swa.rope_tables(8, 64), "swa_rope_apply": lambda: swa.rope_apply(k, k, rope),
        "swa_kv4_plan": lambda: swa.kv4_plan(lens, lens, table, torch.zeros(4, **i32), torch.zeros(1, **i32), page=16, n_pages=4, n_tokens=3),
        "swa_kv4_append": lambda: swa.kv4_append(cache, k, k, slot), "swa_kv4_read": lambda: swa.kv4_read(cache, slot),
        "swa_kv4_attn": lambda: swa.kv4_attention(cache, q, table, lens, workspace=ws)}


@pytest.mark.parametrize("name", NAMES)
def test_a_failed_call_is_told_and_not_made_again(name, bind):
    call, made = calls()[name], []
    bind(name, lambda *a: made.append(1) or swa.SWA_ERR_CUDA)
    with pytest.raises(swa.SwaError, match="CUDA") as e:
        call()
    assert e.value.status == swa.SWA_ERR_CUDA and name in str(e.value) and made == [1]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("status", [swa.SWA_ERR_INVALID_ARG, swa.SWA_ERR_UNSUPPORTED, swa.SWA_ERR_WORKSPACE])
def test_a_call_that_is_refused_before_its_launch_goes_the_long_way(name, status, bind):
    call, made = calls()[name], []
    call()
    bind(name, lambda *a: made.append(1) or status)
    call()             # the library itself takes it
    assert made == [1]


def test_rotation_in_place_that_meets_an_older_error_turns_once(bind):
    # the launch goes through, and what is reported is an error left by other code
    lib = swa.load("bf16")
    rope = swa.rope_tables(9, 64)
    q, k = (randn(i, 1, 9, 2, 64, dtype=torch.bfloat16).to(dev()) for i in (1, 2))
    want = swa.rope_apply(q, k, rope)
    bind("swa_rope_apply", lambda *a: lib.swa_rope_apply(*a) or swa.SWA_ERR_CUDA)
    with pytest.raises(swa.SwaError):
        swa.rope_apply(q, k, rope, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


STUB = r"""
#include <unistd.h>
volatile int entered = 0, go = 0, waited = 0;
int stub(const void* a, int b, int c, void* d, void* e, void* f) {
  entered = 1;
  for (int i = 0; i < 5000 && !go; ++i) usleep(1000);   /* at most 5 s */
  waited = go ? 1 : -1;
  return 0;
}
"""


def test_other_threads_run_beside_a_call(bind, tmp_path):
    # a call that waits, as one does on a full launch queue, until another
    # Python thread has let it go on
    (tmp_path / "stub.c").write_text(STUB)
    so = os.fspath(tmp_path / "stub.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", so, os.fspath(tmp_path / "stub.c")], check=True)
    lib = ctypes.CDLL(so)
    entered, go, waited = (ctypes.c_int.in_dll(lib, n) for n in ("entered", "go", "waited"))
    bind("swa_rope_tables", lib.stub)

    def let_go():
        while not entered.value and time.monotonic() < end:
            time.sleep(0.001)
        go.value = 1

    end = time.monotonic() + 20
    t = threading.Thread(target=let_go)
    t.start()
    swa.rope_tables(8, 64)
    t.join()
    assert waited.value == 1, "the call held the interpreter"


def test_an_argument_without_a_truth_value_stops_the_call(bind):
    made = []
    bind("swa_rope_apply", lambda *a: made.append(1) or swa.SWA_OK)
    rope = swa.rope_tables(9, 64)
    q = randn(1, 1, 9, 2, 64, dtype=torch.bfloat16).to(dev())
    before = q.clone()
    for kw in (dict(inverse=torch.ones(2)), dict(interleaved=torch.ones(2))):
        with pytest.raises(RuntimeError, match="ambiguous"):
            swa.rope_apply(q, None, rope, out=(q, None), **kw)
    assert not made and torch.equal(q, before)

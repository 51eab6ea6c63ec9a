"""Host side of the decode calls' binding: what an import loads, and which
build of the short way (csrc/py_fast.cpp) is taken; sizes that the calls take.
Nothing here runs on a GPU."""

import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

import sliding_window_gqa_qk_gb300 as swa
from sliding_window_gqa_qk_gb300 import build as swa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="session", autouse=True)
def built_libraries():
    swa_build.build()


def run(code, **kw):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, check=True, **kw).stdout


def test_an_import_maps_no_library_of_the_package():
    code = ("import os, sliding_window_gqa_qk_gb300 as swa\n"
            "mapped = lambda: sorted({os.path.basename(x.split()[-1]) for x in open('/proc/self/maps') if os.path.dirname(swa.__file__) in x})\n"
            "print(mapped()); swa.load('bf16'); print(mapped(), swa._fast is not None)")
    before, after = run(code).splitlines()
    assert before == "[]"
    assert "libswaattn.so" in after and "_fast" in after and after.endswith("True")


def test_the_short_way_is_that_of_this_torch_and_python(monkeypatch):
    here = swa_build.fast_path()
    assert os.path.exists(here)
    torch_version = torch.__version__
    monkeypatch.setattr("torch.__version__", torch_version + ".other")
    assert swa_build.fast_path() != here and not os.path.exists(swa_build.fast_path())
    monkeypatch.setattr("torch.__version__", torch_version)
    monkeypatch.setattr(swa_build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert swa_build.fast_path() != here and not os.path.exists(swa_build.fast_path())
    # one built for another torch, or without a name for any, is left alone
    code = ("import torch\ntorch.__version__ += '.other'\nimport sliding_window_gqa_qk_gb300 as swa\nswa.load('bf16')\n"
            "print(swa._fast)\nprint([x for x in open('/proc/self/maps') if '_fast' in x and 'gb300' in x])")
    assert run(code).split() == ["None", "[]"]


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

A = 1 << 20


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses would be used")
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_the_row_calls_take_any_number_of_tokens(kind):
    # what the same calls of a few tokens end with on a machine without a GPU
    cache, rope = swa.swa_kv4_cache(A, 10, 32), swa.swa_rope(A, A, 1 << 23, 64, 0)

    def ends(**kw):
        p = swa.make_params(**dict(dict(B=2, T=3, Hq=4, Hkv=2, d=128), **kw))
        return (swa.swa_rope_apply(p, rope, A, A, A, A, A, kind=kind), swa.swa_kv4_append(p, None, cache, rope, A, A, None, None, None, None, A, A, kind=kind),
                swa.swa_kv4_read(p, cache, A, A, A, kind=kind))

    few = ends()
    assert few[0] != swa.SWA_OK and len(set(few)) == 1
    for kw in (dict(B=16384, T=1), dict(B=104000, T=1, Hq=3, Hkv=3), dict(B=2 ** 31 - 1, T=1, Hq=1, Hkv=1), dict(B=1, T=(1 << 22) + 1),
               dict(B=40000, T=2, Hq=65535, Hkv=1)):
        assert ends(**kw) == few, kw
        assert swa.swa_kv4_cache_size(swa.make_params(**dict(dict(B=2, T=3, Hq=4, Hkv=2, d=128), **kw)), 10, 32, kind) > 0
    assert set(ends(B=1, T=1, Hq=65536)) == {swa.SWA_ERR_UNSUPPORTED}
    # the attention counts requests and heads in its grid
    attn = lambda **kw: swa.swa_kv4_attn(swa.make_params(T=1, d=64, **kw), None, cache, None, A, None, A, 4, A, A, A, A, 1 << 40, kind=kind)   # noqa: E731
    assert attn(B=65536, Hq=1, Hkv=1) == swa.SWA_ERR_UNSUPPORTED and attn(B=65535, Hq=1, Hkv=1) == few[0]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses would be used")
def test_new_outputs_of_a_rotation_are_no_inputs():
    p, rope = swa.make_params(B=2, T=3, Hq=4, Hkv=2, d=128), swa.swa_rope(A, A, 64, 64, 0)
    new = swa.SWA_ROPE_NEW_OUTPUTS
    apply = lambda *args: swa.swa_rope_apply(p, rope, None, *args, kind="bf16")   # noqa: E731
    plain = apply(A, A, 2 * A, 3 * A, 0)
    for mode in (new, new + 1):
        assert apply(A, A, 2 * A, 3 * A, mode) == plain
        for q, k, qo, ko in ((A, A, A, 3 * A), (A, A, 2 * A, A), (None, A, None, A), (A, None, A, None)):
            assert apply(q, k, qo, ko, mode) == swa.SWA_ERR_INVALID_ARG
        assert apply(A, None, 2 * A, None, mode) == plain
    for mode in (2, 3, new + 2, 8, -1):
        assert apply(A, A, 2 * A, 3 * A, mode) == swa.SWA_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# Arithmetic
# ---------------------------------------------------------------------------

OVER_15 = r"""
#include <math.h>
#include <stdint.h>
#include <string.h>
%s
static float at(uint32_t bits) { float f; memcpy(&f, &bits, 4); return f; }
/* wrong quotients of every fp32 number of `n` binades from exponent e0 on */
extern "C" long wrong(int e0, int n) {
  long bad = 0;
  for (uint32_t b = (uint32_t)e0 << 23; b < (uint32_t)(e0 + n) << 23; ++b) bad += over_15(at(b)) != at(b) / 15.0f;
  return bad;
}
"""


def test_a_span_over_15_is_correctly_rounded(tmp_path):
    # the kernel's own function, compiled for the host: every span of the
    # binades that a step's fraction can come from (the quotient's takes in
    # two), at the ends of the range of steps that do not count as 0 and at 1
    source = open(os.path.join(ROOT, "sliding_window_gqa_qk_gb300", "csrc", "kv4.cuh")).read()
    code = re.search(r"__device__ __forceinline__ (float over_15\(float x\) \{.*?\n\})", source, re.S).group(1)
    (tmp_path / "over.cpp").write_text(OVER_15 % code)
    so = os.fspath(tmp_path / "over.so")
    subprocess.run(["g++", "-O2", "-ffp-contract=off", "-shared", "-fPIC", "-o", so, os.fspath(tmp_path / "over.cpp")], check=True)
    wrong = ctypes.CDLL(so).wrong
    wrong.restype = ctypes.c_long
    for e0 in (127 - 116, 126, 253):       # 15e-36 is 2^-115.7
        assert wrong(e0, 2) == 0, e0

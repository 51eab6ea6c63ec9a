"""Host side of the decode calls' binding: what an import loads, and which
build of the short way (csrc/py_fast.cpp) is taken. Nothing here runs on a GPU."""

import os
import subprocess
import sys

import pytest

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
    torch_version = __import__("torch").__version__
    monkeypatch.setattr("torch.__version__", torch_version + ".other")
    assert swa_build.fast_path() != here and not os.path.exists(swa_build.fast_path())
    monkeypatch.setattr("torch.__version__", torch_version)
    monkeypatch.setattr(swa_build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert swa_build.fast_path() != here and not os.path.exists(swa_build.fast_path())
    # one built for another torch, or without a name for any, is left alone
    code = ("import torch\ntorch.__version__ += '.other'\nimport sliding_window_gqa_qk_gb300 as swa\nswa.load('bf16')\n"
            "print(swa._fast)\nprint([x for x in open('/proc/self/maps') if '_fast' in x and 'gb300' in x])")
    assert run(code).split() == ["None", "[]"]

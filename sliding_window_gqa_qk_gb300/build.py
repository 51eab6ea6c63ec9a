"""Builds the two shared libraries of the package in-tree with nvcc:

  libswaattn.so       bf16 tensors, tcgen05 kernels (the product path)
  libswaattn_fp32.so  fp32 tensors, SIMT debug kernels

Both come from csrc/swa_attn.cu, compiled for sm_103a only. And, with the host
compiler against the installed torch:

  _fast.*.so          the binding's short way into the decode calls
                      (csrc/py_fast.cpp); the binding works without it, only
                      slower, so a failure to build it is a warning. It reads
                      Python's and torch's objects by their headers, so its
                      name holds the versions of both: under another torch or
                      Python it is not there, and is built again.
"""

from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")

LIBS = {
    "bf16": ("libswaattn.so", []),
    "fp32": ("libswaattn_fp32.so", ["-DSWA_ELEM_FP32"]),
}

NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def lib_path(kind: str) -> str:
    return os.path.join(PKG, LIBS[kind][0])


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in _sources())


def fast_path() -> str:
    """The short way's module as built for this Python and this torch."""
    import torch
    tag = re.sub(r"[^A-Za-z0-9]+", "_", torch.__version__)
    return os.path.join(PKG, f"_fast.{sysconfig.get_config_var('SOABI')}.torch_{tag}.so")


def _fast_cmd(out: str, nvcc: str):
    """The host compiler's command for the short way."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), "/usr/local/cuda/include"]
    return [shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + i for i in include), "-o", out,
            os.path.join(CSRC, "py_fast.cpp"), "-L" + os.path.join(base, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python",
            "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> None:
    """Compiles every library that is missing or older than its sources,
    in parallel. Raises RuntimeError with nvcc's output on failure."""
    nvcc = nvcc_path()
    procs = []
    for kind, (name, defs) in LIBS.items():
        out = os.path.join(PKG, name)
        if not force and not _stale(out):
            continue
        tmp = out + ".tmp"
        cmd = [nvcc, *NVCC_FLAGS, *defs, "-o", tmp, os.path.join(CSRC, "swa_attn.cu")]
        if verbose:
            print(" ".join(cmd))
        procs.append((out, tmp, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)))
    fast = None
    try:
        fast = fast_path()
        if force or _stale(fast):
            cmd = _fast_cmd(fast + ".tmp", nvcc)
            if verbose:
                print(" ".join(cmd))
            procs.append((fast, fast + ".tmp", subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    except (OSError, ImportError, AttributeError) as e:
        warnings.warn(f"the short way (_fast) is not built: {e}")
    errors = []
    for out, tmp, p in procs:
        log, _ = p.communicate()
        if p.returncode != 0 and out == fast:
            warnings.warn("the short way (_fast) is not built:\n" + log[-2000:])
        elif p.returncode != 0:
            errors.append(f"{os.path.basename(out)}:\n{log}")
        else:
            os.replace(tmp, out)
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))


if __name__ == "__main__":
    build(force=True, verbose=True)

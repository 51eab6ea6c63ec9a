"""Python binding of the GB300 attention-block library (C ABI in
``include/swa_attn.h``).

The functions named ``swa_*`` mirror the C entry points one to one and only
marshal arguments (tensor pointers, the CUDA stream, the parameter struct).
``attention_forward`` / ``attention_backward`` allocate outputs and the
workspace with PyTorch and call them. Every computation runs in the CUDA
library; if the shared library is missing, loading it raises.

Two libraries share the symbols: ``libswaattn.so`` (bf16 tensors, tcgen05
kernels) and ``libswaattn_fp32.so`` (fp32 tensors, SIMT debug kernels). The
binding picks the one matching the dtype of ``q``.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional

import torch

from . import build as _build


class _Unloaded:
    """Stands for the short way into the decode calls (csrc/py_fast.cpp) until
    load() brings it in with the library it leads to: leaves every call to the
    long way, and keeps the import of the package free of compiled code."""

    def __getattr__(self, name):
        return lambda *args: None


_fast = _Unloaded()      # None once load() finds that it is not built: everything works without it

__all__ = [
    "swa_params", "SwaError", "load",
    "swa_attn_workspace_size", "swa_attn_workspace_init", "swa_attn_fwd", "swa_attn_bwd",
    "swa_attn_fwd_ex", "swa_attn_bwd_ex",
    "swa_attn_fwd_noalloc",
    "swa_block_weights", "swa_block_workspace_size", "swa_block_fwd", "swa_block_bwd",
    "make_block_weights", "make_block_extras",
    "swa_attn_check_status", "swa_sssl_window", "swa_has_ve", "swa_strerror",
    "swa_build_info", "attention_forward", "attention_backward", "make_params",
    "swa_rope", "swa_rope_freq", "swa_kv4_cache", "swa_rope_tables", "swa_rope_apply",
    "swa_kv4_cache_size", "swa_kv4_plan", "swa_kv4_append", "swa_kv4_read",
    "swa_kv4_workspace_size", "swa_kv4_workspace_init", "swa_kv4_attn",
    "rope_tables", "rope_apply", "new_kv4_cache", "new_kv4_workspace", "kv4_plan", "kv4_append",
    "kv4_read", "kv4_attention",
    "swa_kv4_tree", "swa_kv4_tree_attn", "swa_kv4_move", "swa_rms_norm", "swa_rms_norm_workspace_size", "swa_rms_norm_bwd",
    "swa_w4_size", "swa_w4_pack", "swa_w4_unpack", "swa_w4_linear", "swa_kv4_weights", "swa_kv4_block_workspace_size",
    "swa_kv4_block", "new_kv4_block_workspace", "kv4_block",
    "kv4_tree", "kv4_tree_attention", "kv4_move", "rms_norm", "rms_norm_backward", "w4_pack", "w4_unpack", "w4_linear",
    "SWA_OK", "SWA_ERR_INVALID_ARG", "SWA_ERR_UNSUPPORTED", "SWA_ERR_CUDA", "SWA_ERR_TIMEOUT",
    "SWA_ERR_WORKSPACE", "SWA_ERR_DEVICE_CHECK", "SWA_REUSE_PROLOGUE", "SWA_BWD_STAGE_PRE",
    "SWA_BWD_STAGE_MAIN", "SWA_BWD_STAGE_POST",
]

SWA_OK = 0
SWA_ERR_INVALID_ARG = 1
SWA_ERR_UNSUPPORTED = 2
SWA_ERR_CUDA = 3
SWA_ERR_TIMEOUT = 4
SWA_ERR_WORKSPACE = 5
SWA_ERR_DEVICE_CHECK = 6

SWA_REUSE_PROLOGUE = 1
SWA_BWD_STAGE_PRE = 2
SWA_BWD_STAGE_MAIN = 4
SWA_BWD_STAGE_POST = 8


def _int32(value):
    """value, where it fits 32 bits: ctypes would cut it to them without a word."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{value} does not fit 32 bits")
    return value


class _Int(ctypes.c_int):
    """An int argument of the library."""

    @classmethod
    def from_param(cls, value):
        return value if isinstance(value, ctypes.c_int) else ctypes.c_int(_int32(value))


_init = ctypes.Structure.__init__


class _Struct(ctypes.Structure):
    def __init_subclass__(cls):
        cls._ints = {name: i for i, (name, kind) in enumerate(cls._fields_) if kind is ctypes.c_int}
        cls._at = tuple(cls._ints.values())

    def __init__(self, *args, **kw):
        if kw or len(args) < len(self._fields_):
            for name, i in self._ints.items():
                _int32(args[i] if i < len(args) else kw.get(name, 0))
            _init(self, *args, **kw)
        else:                       # (in a hurry: the calls of a decode step make four of these)
            for i in self._at:
                if not -0x80000000 <= args[i] <= 0x7fffffff:
                    _int32(args[i])
            _init(self, *args)


class swa_params(_Struct):
    _fields_ = [
        ("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("d", ctypes.c_int), ("window", ctypes.c_int), ("causal", ctypes.c_int),
        ("softmax_scale", ctypes.c_float), ("eps", ctypes.c_float),
        ("ve_scale", ctypes.c_float), ("vocab", ctypes.c_int),
    ]


class SwaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {swa_strerror(status)} (status {status})")
        self.status = status


class swa_extras(_Struct):
    """Extras of the _ex entry points: rotary tables, the learned
    value-embedding gate and the pipeline-wait limit (see include/swa_attn.h)."""
    _fields_ = [("rope_cos", ctypes.c_void_p), ("rope_sin", ctypes.c_void_p), ("rope_rows", ctypes.c_int),
                ("gate_x", ctypes.c_void_p), ("gate_x_stride", ctypes.c_longlong),
                ("gate_w", ctypes.c_void_p), ("gate_ch", ctypes.c_int),
                ("d_gate_w", ctypes.c_void_p), ("d_gate_x", ctypes.c_void_p),
                ("wait_limit_ns", ctypes.c_ulonglong)]


class swa_block_weights(_Struct):
    """Weights of the block calls: model width C and the four projection
    matrices in the torch.nn.Linear layout (see include/swa_attn.h)."""
    _fields_ = [("C", ctypes.c_int), ("wq", ctypes.c_void_p), ("wk", ctypes.c_void_p),
                ("wv", ctypes.c_void_p), ("wo", ctypes.c_void_p)]


class swa_rope(_Struct):
    """Rotary tables of the rope and kv4 calls (see include/swa_attn.h)."""
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int),
                ("rot", ctypes.c_int), ("interleaved", ctypes.c_int)]


class swa_rope_freq(_Struct):
    """Frequencies of swa_rope_tables (see include/swa_attn.h)."""
    _fields_ = [("rot", ctypes.c_int), ("scaling", ctypes.c_int)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "orig_len", "slow", "fast", "amplitude")]


class swa_kv4_cache(_Struct):
    """A 4-bit paged cache: device buffer, pages, tokens per page."""
    _fields_ = [("data", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("page", ctypes.c_int)]


class swa_kv4_weights(_Struct):
    """Packed weights of swa_kv4_block (see include/swa_attn.h)."""
    _fields_ = [("C", ctypes.c_int)] + [(n, ctypes.c_void_p) for n in ("wq", "wk", "wv", "wo")]


_LIBS: dict = {}
_vp = ctypes.c_void_p


def _load_fast() -> None:
    global _fast
    if isinstance(_fast, _Unloaded):
        path = _build.fast_path()
        spec = importlib.util.spec_from_file_location(__name__ + "._fast", path)
        try:
            if not os.path.exists(path):
                raise ImportError(path)
            _fast = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_fast)
        except ImportError:
            _fast = None


def load(kind: str = "bf16") -> ctypes.CDLL:
    """The ctypes handle of the bf16 or fp32 library (loaded once)."""
    if kind in _LIBS:
        return _LIBS[kind]
    path = _build.lib_path(kind)
    if not os.path.exists(path):
        raise RuntimeError(
            f"{os.path.basename(path)} is not built; run sliding_window_gqa_qk_gb300.build.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(swa_params)
    lib.swa_attn_workspace_size.argtypes = [P, ctypes.c_int]
    lib.swa_attn_workspace_size.restype = ctypes.c_size_t
    lib.swa_attn_workspace_init.argtypes = [_vp, ctypes.c_size_t, _vp]
    lib.swa_attn_workspace_init.restype = ctypes.c_int
    lib.swa_attn_fwd.argtypes = [P] + [_vp] * 11 + [ctypes.c_size_t, ctypes.c_uint, _vp]
    lib.swa_attn_fwd.restype = ctypes.c_int
    lib.swa_attn_bwd.argtypes = [P] + [_vp] * 18 + [ctypes.c_size_t, ctypes.c_uint, _vp]
    lib.swa_attn_bwd.restype = ctypes.c_int
    R = ctypes.POINTER(swa_extras)
    lib.swa_attn_fwd_ex.argtypes = [P, R] + [_vp] * 11 + [ctypes.c_size_t, ctypes.c_uint, _vp]
    lib.swa_attn_fwd_ex.restype = ctypes.c_int
    lib.swa_attn_bwd_ex.argtypes = [P, R] + [_vp] * 18 + [ctypes.c_size_t, ctypes.c_uint, _vp]
    lib.swa_attn_bwd_ex.restype = ctypes.c_int
    lib.swa_attn_fwd_noalloc.argtypes = [P] + [_vp] * 10 + [_vp]
    lib.swa_attn_fwd_noalloc.restype = ctypes.c_int
    lib.swa_attn_step_host_size.argtypes = [P]
    lib.swa_attn_step_host_size.restype = ctypes.c_size_t
    lib.swa_attn_step_host.argtypes = [P, R] + [_vp] * 18 + [ctypes.c_size_t, _vp]
    lib.swa_attn_step_host.restype = ctypes.c_int
    W = ctypes.POINTER(swa_block_weights)
    lib.swa_block_workspace_size.argtypes = [P, ctypes.c_int, ctypes.c_int]
    lib.swa_block_workspace_size.restype = ctypes.c_size_t
    lib.swa_block_fwd.argtypes = [P, R, W] + [_vp] * 7 + [ctypes.c_size_t, _vp]
    lib.swa_block_fwd.restype = ctypes.c_int
    lib.swa_block_bwd.argtypes = [P, R, W] + [_vp] * 15 + [ctypes.c_size_t, _vp]
    lib.swa_block_bwd.restype = ctypes.c_int
    C, F, I, L, Z = (ctypes.POINTER(swa_kv4_cache), ctypes.POINTER(swa_rope), _Int, ctypes.c_longlong, ctypes.c_size_t)
    for name, args in (
            ("swa_rope_tables", [ctypes.POINTER(swa_rope_freq), I, I, _vp, _vp, _vp]),
            ("swa_rope_apply", [P, F] + [_vp] * 5 + [I, _vp, Z, _vp]),
            ("swa_kv4_plan", [I] * 4 + [_vp] * 4 + [I, _vp, I] + [_vp] * 7 + [Z, _vp]),
            ("swa_kv4_append", [P, R, C, F] + [_vp] * 9 + [Z, _vp]),
            ("swa_kv4_read", [P, C] + [_vp] * 4 + [Z, _vp]),
            ("swa_kv4_workspace_init", [_vp, Z, _vp]),
            ("swa_kv4_attn", [P, R, C, F, _vp, _vp, _vp, I] + [_vp] * 4 + [Z, _vp]),
            ("swa_kv4_tree", [I] * 3 + [_vp] * 6 + [Z, _vp]),
            ("swa_kv4_tree_attn", [P, R, C, F, I, I, _vp, _vp, _vp, I] + [_vp] * 7 + [Z, _vp]),
            ("swa_kv4_move", [P, C] + [_vp] * 3 + [Z, _vp]),
            ("swa_kv4_block", [P, R, C, F, ctypes.POINTER(swa_kv4_weights), I, I] + [_vp] * 12 + [I] + [_vp] * 3 + [Z, _vp]),
            ("swa_rms_norm", [L, I, ctypes.c_float] + [_vp] * 9),
            ("swa_rms_norm_bwd", [L, I] + [_vp] * 8 + [Z, _vp]),
            ("swa_w4_pack", [I, I] + [_vp] * 3),
            ("swa_w4_unpack", [I, I] + [_vp] * 3),
            ("swa_w4_linear", [I] * 3 + [_vp] * 5 + [_vp, Z, _vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ctypes.c_int
    for name, args in (("swa_kv4_cache_size", [P, I, I]), ("swa_kv4_workspace_size", [P, I, I]),
                       ("swa_rms_norm_workspace_size", [L, I]), ("swa_w4_size", [I, I]), ("swa_kv4_block_workspace_size", [P, I, I])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = Z
    lib.swa_attn_check_status.argtypes = [_vp, _vp]
    lib.swa_attn_check_status.restype = ctypes.c_int
    lib.swa_sssl_window.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_char_p, ctypes.c_int]
    lib.swa_sssl_window.restype = ctypes.c_int
    lib.swa_has_ve.argtypes = [ctypes.c_int, ctypes.c_int]
    lib.swa_has_ve.restype = ctypes.c_int
    lib.swa_strerror.argtypes = [ctypes.c_int]
    lib.swa_strerror.restype = ctypes.c_char_p
    lib.swa_build_info.argtypes = []
    lib.swa_build_info.restype = ctypes.c_char_p
    _LIBS[kind] = lib
    _load_fast()
    if _fast is not None:
        _fast.raises(SwaError)
        _fast.bind(0 if kind == "bf16" else 1, *(
            ctypes.cast(getattr(lib, f), _vp).value for f in (
                "swa_rope_tables", "swa_rope_apply", "swa_kv4_plan", "swa_kv4_append", "swa_kv4_read", "swa_kv4_attn")))
        _fast.bind_more(0 if kind == "bf16" else 1, *(
            ctypes.cast(getattr(lib, f), _vp).value for f in (
                "swa_rms_norm", "swa_rms_norm_workspace_size", "swa_rms_norm_bwd", "swa_w4_linear", "swa_kv4_tree",
                "swa_kv4_tree_attn", "swa_kv4_move")))
    return lib


def _kind_of(t: Optional[torch.Tensor]) -> str:
    if t is not None and t.dtype == torch.float32:
        return "fp32"
    return "bf16"


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_params(B, T, Hq, Hkv, d, window=-1, causal=True, softmax_scale=0.0, eps=1e-6,
                ve_scale=0.5, vocab=0) -> swa_params:
    return swa_params(int(B), int(T), int(Hq), int(Hkv), int(d), int(window), int(bool(causal)),
                      float(softmax_scale), float(eps), float(ve_scale), int(vocab))


# ---------------------------------------------------------------------------
# One-to-one wrappers of the C entry points
# ---------------------------------------------------------------------------

def swa_attn_workspace_size(p: swa_params, for_backward: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_attn_workspace_size(ctypes.byref(p), int(for_backward)))


def swa_attn_workspace_init(ws, ws_bytes=None, stream=None, kind: str = "bf16") -> int:
    n = ws.numel() if ws_bytes is None else ws_bytes
    return int(load(kind).swa_attn_workspace_init(_ptr(ws), n, _stream(stream)))


def swa_attn_fwd(p, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, ws, ws_bytes=None, flags=0,
                 stream=None, kind=None) -> int:
    kind = kind or _kind_of(q)
    n = ws.numel() if ws_bytes is None else ws_bytes
    return int(load(kind).swa_attn_fwd(
        ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(ve_gate), _ptr(o), _ptr(lse), _ptr(ws), n, int(flags), _stream(stream)))


def swa_attn_bwd(p, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, dO, dq, dk, dv, dgq, dgk, dve,
                 ws, ws_bytes=None, flags=0, stream=None, kind=None) -> int:
    kind = kind or _kind_of(q)
    n = ws.numel() if ws_bytes is None else ws_bytes
    return int(load(kind).swa_attn_bwd(
        ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(ve_gate), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dgq),
        _ptr(dgk), _ptr(dve), _ptr(ws), n, int(flags), _stream(stream)))


def make_extras(rope=None, gate_x=None, gate_w=None, d_gate_w=None, d_gate_x=None,
                wait_limit_ns: int = 0) -> swa_extras:
    """swa_extras from device tensors: rope = (cos, sin) fp32 [rows, d/2] or
    None; gate_x [B, T, >= C] rows (its row stride is taken from the tensor),
    gate_w fp32 [Hkv, C] or None; backward outputs d_gate_w [Hkv, C],
    d_gate_x [B, T, C] (fp32) or None; wait_limit_ns the time limit of one
    pipeline wait of the kernels (0: the library's default)."""
    e = swa_extras()
    e.wait_limit_ns = int(wait_limit_ns)
    if rope is not None:
        e.rope_cos, e.rope_sin, e.rope_rows = _ptr(rope[0]), _ptr(rope[1]), int(rope[0].shape[0])
    if gate_w is not None:
        if gate_x.stride(-1) != 1 or gate_x.dim() != 3 or gate_x.stride(0) != gate_x.shape[1] * gate_x.stride(1):
            raise ValueError("gate_x must be [B, T, *] with unit channel stride and packed rows")
        e.gate_x = gate_x.data_ptr()
        e.gate_x_stride = int(gate_x.stride(1))
        e.gate_w = _ptr(gate_w)
        e.gate_ch = int(gate_w.shape[1])
        e.d_gate_w = _ptr(d_gate_w)
        e.d_gate_x = _ptr(d_gate_x)
    return e


def swa_attn_fwd_ex(p, ex, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, ws, ws_bytes=None,
                    flags=0, stream=None, kind=None) -> int:
    kind = kind or _kind_of(q)
    n = ws.numel() if ws_bytes is None else ws_bytes
    ep = None if ex is None else ctypes.byref(ex)
    return int(load(kind).swa_attn_fwd_ex(
        ctypes.byref(p), ep, _ptr(q), _ptr(k), _ptr(v), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(ve_gate), _ptr(o), _ptr(lse), _ptr(ws), n, int(flags), _stream(stream)))


def swa_attn_bwd_ex(p, ex, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, dO, dq, dk, dv, dgq, dgk,
                    dve, ws, ws_bytes=None, flags=0, stream=None, kind=None) -> int:
    kind = kind or _kind_of(q)
    n = ws.numel() if ws_bytes is None else ws_bytes
    ep = None if ex is None else ctypes.byref(ex)
    return int(load(kind).swa_attn_bwd_ex(
        ctypes.byref(p), ep, _ptr(q), _ptr(k), _ptr(v), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(ve_gate), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dgq),
        _ptr(dgk), _ptr(dve), _ptr(ws), n, int(flags), _stream(stream)))


def swa_attn_step_host_size(p: swa_params, kind: str = "bf16") -> int:
    return int(load(kind).swa_attn_step_host_size(ctypes.byref(p)))


def swa_attn_step_host(p, ex, q, k, v, gq, gk, ve, tok, ve_gate, dO, o, lse, dq, dk, dv, dgq, dgk,
                       dve, buf, buf_bytes=None, stream=None, kind=None) -> int:
    """One forward + backward with host tensors (inputs and outputs on the
    CPU, ideally pinned) and a device buffer of swa_attn_step_host_size
    bytes; enqueued on `stream`, returns without waiting."""
    kind = kind or _kind_of(q)
    n = buf.numel() if buf_bytes is None else buf_bytes
    ep = None if ex is None else ctypes.byref(ex)
    return int(load(kind).swa_attn_step_host(
        ctypes.byref(p), ep, _ptr(q), _ptr(k), _ptr(v), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(ve_gate), _ptr(dO), _ptr(o), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dgq),
        _ptr(dgk), _ptr(dve), _ptr(buf), n, _stream(stream)))


def new_step_host_buffer(p: swa_params, device, kind: str, stream=None):
    """A device buffer for swa_attn_step_host, initialised."""
    n = swa_attn_step_host_size(p, kind)
    if n == 0:
        raise SwaError(SWA_ERR_INVALID_ARG, "step buffer size")
    buf = torch.empty(n, dtype=torch.uint8, device=device)
    _check(swa_attn_workspace_init(buf, n, stream, kind), "step buffer init")
    return buf


def swa_attn_fwd_noalloc(p, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, stream=None,
                         kind=None) -> int:
    """Forward whose scratch is the library's fixed device array (no
    workspace argument, nothing allocated); see include/swa_attn.h."""
    kind = kind or _kind_of(q)
    return int(load(kind).swa_attn_fwd_noalloc(
        ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(ve_gate), _ptr(o), _ptr(lse), _stream(stream)))


def make_block_weights(wq, wk, wv, wo) -> swa_block_weights:
    """swa_block_weights from device tensors wq [Hq*d, C], wk, wv [Hkv*d, C],
    wo [C, Hq*d] (the model width C is taken from wq)."""
    return swa_block_weights(int(wq.shape[1]), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(wo))


def make_block_extras(rope=None, gate_w=None, d_gate_w=None) -> swa_extras:
    """swa_extras of the block calls: rope = (cos, sin) fp32 [rows, d/2] or
    None; gate_w fp32 [Hkv, C] (the block feeds the gate its normed input);
    d_gate_w fp32 [Hkv, C] backward output or None."""
    e = make_extras(rope)
    if gate_w is not None:
        e.gate_w = _ptr(gate_w)
        e.gate_ch = int(gate_w.shape[1])
        e.d_gate_w = _ptr(d_gate_w)
    return e


def swa_block_workspace_size(p: swa_params, C: int, for_backward: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_block_workspace_size(ctypes.byref(p), int(C), int(for_backward)))


def swa_block_fwd(p, ex, w, x, gq, gk, ve, tok, out, ws, ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(x)
    n = ws.numel() if ws_bytes is None else ws_bytes
    ep = None if ex is None else ctypes.byref(ex)
    return int(load(kind).swa_block_fwd(
        ctypes.byref(p), ep, ctypes.byref(w), _ptr(x), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(out), _ptr(ws), n, _stream(stream)))


def swa_block_bwd(p, ex, w, x, gq, gk, ve, tok, dout, dx, dwq, dwk, dwv, dwo, dgq, dgk, dve, ws,
                  ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(x)
    n = ws.numel() if ws_bytes is None else ws_bytes
    ep = None if ex is None else ctypes.byref(ex)
    return int(load(kind).swa_block_bwd(
        ctypes.byref(p), ep, ctypes.byref(w), _ptr(x), _ptr(gq), _ptr(gk), _ptr(ve), _ptr(tok),
        _ptr(dout), _ptr(dx), _ptr(dwq), _ptr(dwk), _ptr(dwv), _ptr(dwo), _ptr(dgq), _ptr(dgk),
        _ptr(dve), _ptr(ws), n, _stream(stream)))


def _ref(s):
    return None if s is None else ctypes.byref(s)


def _ws_bytes(ws, ws_bytes):
    return ws_bytes if ws_bytes is not None else (0 if ws is None else ws.numel())


def swa_rope_tables(f: swa_rope_freq, first: int, rows: int, cos, sin, stream=None, kind: str = "bf16") -> int:
    return int(load(kind).swa_rope_tables(ctypes.byref(f), int(first), int(rows), _ptr(cos), _ptr(sin), _stream(stream)))


def swa_rope_apply(p, r, pos, q, k, q_out, k_out, inverse=0, ws=None, ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(q if q is not None else k)
    return int(load(kind).swa_rope_apply(
        ctypes.byref(p), _ref(r), _ptr(pos), _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), int(inverse), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_cache_size(p: swa_params, n_pages: int, page: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_cache_size(ctypes.byref(p), int(n_pages), int(page)))


def swa_kv4_plan(n_pages, page, B, max_pages, lens, new_lens, table, free_pages, n_free, free_head, n_tokens, slot, pos,
                 row, cu, lens_out, head_out, ws=None, ws_bytes=None, stream=None, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_plan(
        n_pages, page, B, max_pages, _ptr(lens), _ptr(new_lens), _ptr(table), _ptr(free_pages), n_free, _ptr(free_head),
        n_tokens, _ptr(slot), _ptr(pos), _ptr(row), _ptr(cu), _ptr(lens_out), _ptr(head_out), _ptr(ws),
        _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_append(p, ex, c, r, k, v, gk, ve, tok, ve_gate, pos, slot, ws=None, ws_bytes=None, stream=None,
                   kind=None) -> int:
    kind = kind or _kind_of(k)
    return int(load(kind).swa_kv4_append(
        ctypes.byref(p), _ref(ex), _ref(c), _ref(r), _ptr(k), _ptr(v), _ptr(gk), _ptr(ve), _ptr(tok), _ptr(ve_gate),
        _ptr(pos), _ptr(slot), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_read(p, c, slot, k_out, v_out, ws=None, ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(k_out)
    return int(load(kind).swa_kv4_read(ctypes.byref(p), _ref(c), _ptr(slot), _ptr(k_out), _ptr(v_out), _ptr(ws),
                                       _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_workspace_size(p: swa_params, page: int, max_pages: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_workspace_size(ctypes.byref(p), int(page), int(max_pages)))


def swa_kv4_workspace_init(ws, ws_bytes=None, stream=None, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_workspace_init(_ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_attn(p, ex, c, r, q, gq, table, max_pages, lens, o, lse, ws, ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(q)
    return int(load(kind).swa_kv4_attn(
        ctypes.byref(p), _ref(ex), _ref(c), _ref(r), _ptr(q), _ptr(gq), _ptr(table), int(max_pages), _ptr(lens),
        _ptr(o), _ptr(lse), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_tree(B, n_tokens, max_new, parent, cu, lens, pos, seen, ws=None, ws_bytes=None, stream=None, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_tree(B, n_tokens, max_new, _ptr(parent), _ptr(cu), _ptr(lens), _ptr(pos), _ptr(seen), _ptr(ws),
                                       _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_tree_attn(p, ex, c, r, n_tokens, max_new, q, gq, table, max_pages, lens, cu, pos, seen, o, lse, ws, ws_bytes=None,
                      stream=None, kind=None) -> int:
    kind = kind or _kind_of(q)
    return int(load(kind).swa_kv4_tree_attn(
        ctypes.byref(p), _ref(ex), _ref(c), _ref(r), int(n_tokens), int(max_new), _ptr(q), _ptr(gq), _ptr(table), int(max_pages),
        _ptr(lens), _ptr(cu), _ptr(pos), _ptr(seen), _ptr(o), _ptr(lse), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_move(p, c, src, dst, ws=None, ws_bytes=None, stream=None, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_move(ctypes.byref(p), _ref(c), _ptr(src), _ptr(dst), _ptr(ws), _ws_bytes(ws, ws_bytes),
                                       _stream(stream)))


def swa_rms_norm(rows, C, eps, x, add, gain, h, y, y8, scale, rstd, stream=None, kind=None) -> int:
    kind = kind or _kind_of(x)
    return int(load(kind).swa_rms_norm(int(rows), int(C), float(eps), _ptr(x), _ptr(add), _ptr(gain), _ptr(h), _ptr(y), _ptr(y8),
                                       _ptr(scale), _ptr(rstd), _stream(stream)))


def swa_rms_norm_workspace_size(rows: int, C: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_rms_norm_workspace_size(int(rows), int(C)))


def swa_rms_norm_bwd(rows, C, h, rstd, gain, dy, dh, dx, dgain, ws=None, ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(h)
    return int(load(kind).swa_rms_norm_bwd(int(rows), int(C), _ptr(h), _ptr(rstd), _ptr(gain), _ptr(dy), _ptr(dh), _ptr(dx),
                                           _ptr(dgain), _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_w4_size(N: int, K: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_w4_size(int(N), int(K)))


def swa_w4_pack(N, K, w, w4, stream=None, kind=None) -> int:
    return int(load(kind or _kind_of(w)).swa_w4_pack(int(N), int(K), _ptr(w), _ptr(w4), _stream(stream)))


def swa_w4_unpack(N, K, w4, w, stream=None, kind=None) -> int:
    return int(load(kind or _kind_of(w)).swa_w4_unpack(int(N), int(K), _ptr(w4), _ptr(w), _stream(stream)))


def swa_w4_linear(M, N, K, x, x_scale, w4, add, y, stream=None, kind=None, ws=None, ws_bytes=None) -> int:
    return int(load(kind or _kind_of(y)).swa_w4_linear(int(M), int(N), int(K), _ptr(x), _ptr(x_scale), _ptr(w4), _ptr(add), _ptr(y),
                                                       _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_kv4_block_workspace_size(p: swa_params, C: int, n_tokens: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_kv4_block_workspace_size(ctypes.byref(p), int(C), int(n_tokens)))


def swa_kv4_block(p, ex, c, r, w, n_tokens, max_new, x, add, gain, gq, gk, ve, tok, slot, pos, cu, seen, table, max_pages, lens, out,
                  ws, ws_bytes=None, stream=None, kind=None) -> int:
    kind = kind or _kind_of(x)
    return int(load(kind).swa_kv4_block(
        ctypes.byref(p), _ref(ex), _ref(c), _ref(r), _ref(w), int(n_tokens), int(max_new), _ptr(x), _ptr(add), _ptr(gain), _ptr(gq),
        _ptr(gk), _ptr(ve), _ptr(tok), _ptr(slot), _ptr(pos), _ptr(cu), _ptr(seen), _ptr(table), int(max_pages), _ptr(lens), _ptr(out),
        _ptr(ws), _ws_bytes(ws, ws_bytes), _stream(stream)))


def swa_attn_check_status(ws, stream=None, kind: str = "bf16") -> int:
    return int(load(kind).swa_attn_check_status(_ptr(ws), _stream(stream)))


def swa_sssl_window(layer: int, n_layer: int, pattern: str, T: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_sssl_window(layer, n_layer, pattern.encode(), T))


def swa_has_ve(layer: int, n_layer: int, kind: str = "bf16") -> int:
    return int(load(kind).swa_has_ve(layer, n_layer))


def swa_strerror(status: int, kind: str = "bf16") -> str:
    try:
        return load(kind).swa_strerror(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def swa_build_info(kind: str = "bf16") -> str:
    return load(kind).swa_build_info().decode()


# ---------------------------------------------------------------------------
# Convenience calls: allocate outputs / workspace, raise on error
# ---------------------------------------------------------------------------

def _check(status: int, what: str):
    if status != SWA_OK:
        raise SwaError(status, what)


def new_workspace(p: swa_params, for_backward: bool, device, kind: str, stream=None):
    n = swa_attn_workspace_size(p, int(for_backward), kind)
    if n == 0:
        raise SwaError(SWA_ERR_INVALID_ARG, "workspace size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    _check(swa_attn_workspace_init(ws, n, stream, kind), "workspace init")
    return ws


def attention_forward(q, k, v, gq=None, gk=None, *, window: int = -1, causal: bool = True,
                      softmax_scale: float = 0.0, eps: float = 1e-6, ve=None, tok=None,
                      ve_gate=None, ve_scale: float = 0.5, workspace=None, stream=None,
                      rope=None, gate_x=None, gate_w=None):
    """o, lse, workspace = attention_forward(q, k, v, ...). The workspace is
    allocated for the backward too, so it can be passed on to
    ``attention_backward`` with the prologue outputs kept. ``rope``: None or
    (cos, sin) fp32 device tensors [rows >= T, d/2] (rotary before the norm).
    ``gate_x`` [B, T, >= C] and ``gate_w`` fp32 [Hkv, C]: the learned
    value-embedding gate 2 sigmoid(gate_w x[:C]) (then ve_gate must be None)."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    kind = _kind_of(q)
    vocab = ve.shape[0] if ve is not None else 0
    p = make_params(B, T, Hq, Hkv, d, window, causal, softmax_scale, eps, ve_scale, vocab)
    ws = workspace if workspace is not None else new_workspace(p, True, q.device, kind, stream)
    o = torch.empty_like(q)
    lse = torch.empty(B, Hq, T, dtype=torch.float32, device=q.device)
    if rope is None and gate_w is None:
        _check(swa_attn_fwd(p, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, ws, stream=stream),
               "swa_attn_fwd")
    else:
        ex = make_extras(rope, gate_x, gate_w)
        _check(swa_attn_fwd_ex(p, ex, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, ws, stream=stream),
               "swa_attn_fwd_ex")
    return o, lse, ws


def attention_backward(q, k, v, gq, gk, o, lse, dO, *, window: int = -1, causal: bool = True,
                       softmax_scale: float = 0.0, eps: float = 1e-6, ve=None, tok=None,
                       ve_gate=None, ve_scale: float = 0.5, workspace=None,
                       reuse_prologue: bool = False, stream=None, rope=None, gate_x=None,
                       gate_w=None) -> dict:
    """Gradients dq, dk, dv, dgq, dgk, dve (dve None without a VE table) and,
    with the learned gate, dgate_w [Hkv, C] and dgate_x [B, T, C]."""
    B, T, Hq, d = q.shape
    Hkv = k.shape[2]
    kind = _kind_of(q)
    vocab = ve.shape[0] if ve is not None else 0
    p = make_params(B, T, Hq, Hkv, d, window, causal, softmax_scale, eps, ve_scale, vocab)
    ws = workspace if workspace is not None else new_workspace(p, True, q.device, kind, stream)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dgq = torch.empty(d, dtype=torch.float32, device=q.device)
    dgk = torch.empty(d, dtype=torch.float32, device=q.device)
    dve = torch.empty(ve.shape, dtype=torch.float32, device=q.device) if ve is not None else None
    flags = SWA_REUSE_PROLOGUE if (reuse_prologue and workspace is not None) else 0
    out = {"dq": dq, "dk": dk, "dv": dv, "dgq": dgq, "dgk": dgk, "dve": dve, "workspace": ws}
    if rope is None and gate_w is None:
        _check(swa_attn_bwd(p, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, dO, dq, dk, dv, dgq, dgk,
                            dve, ws, flags=flags, stream=stream), "swa_attn_bwd")
    else:
        dgw = dgx = None
        if gate_w is not None:
            dgw = torch.empty(gate_w.shape, dtype=torch.float32, device=q.device)
            dgx = torch.empty(B, T, gate_w.shape[1], dtype=torch.float32, device=q.device)
            out["dgate_w"], out["dgate_x"] = dgw, dgx
        ex = make_extras(rope, gate_x, gate_w, dgw, dgx)
        _check(swa_attn_bwd_ex(p, ex, q, k, v, gq, gk, ve, tok, ve_gate, o, lse, dO, dq, dk, dv, dgq,
                               dgk, dve, ws, flags=flags, stream=stream), "swa_attn_bwd_ex")
    return out


# ---------------------------------------------------------------------------
# Rotary positions and the decode path. These calls check types, shapes and
# devices before they pass addresses on (the C ABI sees addresses only), run
# on the device of their tensors, and allocate their outputs on the stream
# they run on. A decode step is a few microseconds of GPU work, so the ordinary
# case goes through csrc/py_fast.cpp, which returns None for every other that
# it has not launched: the Python below is the whole of each call, the other
# only its short way.
# ---------------------------------------------------------------------------

SWA_ROPE_PLAIN, SWA_ROPE_LINEAR, SWA_ROPE_NTK, SWA_ROPE_BY_PARTS = range(4)
SWA_ROPE_NEW_OUTPUTS = 4
_SCALINGS = {"none": SWA_ROPE_PLAIN, "linear": SWA_ROPE_LINEAR, "ntk": SWA_ROPE_NTK, "by_parts": SWA_ROPE_BY_PARTS}
_NO_ROPE = (None, None)
_F32, _BF16, _I32, _I64, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8
# torch's own lookup of the current stream's handle by device index; the
# public one builds a Stream object each time (2.9 us against 0.1 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _at(name, t, dtype, shape, device):
    """Address of an argument of the calls below after its checks; None passes."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {device} is expected, got "
                         f"{t.dtype}, {tuple(t.shape)}, on {t.device}" + ("" if t.is_contiguous() else ", not contiguous"))
    return t.data_ptr()


def _kind(name, dtype):
    if dtype is _BF16:
        return "bf16"
    if dtype is _F32:
        return "fp32"
    raise ValueError(f"{name}: bf16 or fp32 is expected, got {dtype}")


def _rope_at(rope, interleaved, device):
    if rope is None:
        return None
    cos, sin = rope
    c = _at("rope cos", cos, _F32, cos.shape, device)
    if cos.dim() != 2:
        raise ValueError("rope: two fp32 tensors [rows, rot/2] are expected")
    return swa_rope(c, _at("rope sin", sin, _F32, cos.shape, device), cos.shape[0], 2 * cos.shape[1], 1 if interleaved else 0)


def _ws_at(ws, device):
    """Address and bytes of a workspace; None: none."""
    if ws is None:
        return None, 0
    n = ws.numel()
    return _at("workspace", ws, _U8, (n,), device), n


def _stream_here(device, stream):
    """The current stream's handle, where ``device`` is the current device and
    no other stream is asked for; else None (see _there)."""
    if stream is None and device.type == "cuda" and device.index == torch.cuda.current_device():
        return _raw_stream(device.index)
    return None


def _there(device, stream, call):
    """call() with ``device`` current, and with ``stream`` (a torch stream or a
    raw handle) if one is given, so that what it allocates belongs to the
    stream it runs on."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}, not on a GPU")
    with torch.cuda.device(device):
        if stream is None:
            return call()
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            return call()


def rope_tables(rows: int, rot: int, *, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                orig_len: float = 0.0, slow: float = 1.0, fast: float = 32.0, amplitude: float = 1.0,
                first: int = 0, device=None, stream=None):
    """cos, sin = rope_tables(rows, rot, ...): fp32 tables [rows, rot/2] of the
    rotary angles of positions first .. first + rows - 1, with the frequencies
    scaled for long contexts ("none", "linear", "ntk", "by_parts": the latter
    wants orig_len, the context trained on). They serve ``rope`` of
    attention_forward (rot = d), of rope_apply and of the kv4 calls (first =
    0 there: row t is position t)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling: one of {sorted(_SCALINGS)} is expected, got {scaling!r}")
    if rows < 0 or rot < 0:
        raise ValueError("rows, rot: not below 0")
    if _fast is not None and device is None and stream is None:
        r = _fast.rope_tables(rows, rot, _SCALINGS[scaling], base, factor, orig_len, slow, fast, amplitude, first)
        if r is not None:
            return r
    device = torch.device("cuda" if device is None else device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    st = _stream_here(device, stream)
    if st is None:
        return _there(device, stream, lambda: rope_tables(
            rows, rot, base=base, scaling=scaling, factor=factor, orig_len=orig_len, slow=slow, fast=fast,
            amplitude=amplitude, first=first, device=device))
    f = swa_rope_freq(rot, _SCALINGS[scaling], base, factor, orig_len, slow, fast, amplitude)
    cos = torch.empty((rows, rot // 2), dtype=_F32, device=device)
    sin = torch.empty_like(cos)
    # (an empty tensor has no address; nothing is written then)
    s = load("bf16").swa_rope_tables(f, first, rows, cos.data_ptr() or 256, sin.data_ptr() or 256, st)
    if s:
        raise SwaError(s, "swa_rope_tables")
    return cos, sin


def rope_apply(q, k, rope, *, pos=None, interleaved: bool = False, inverse: bool = False, out=None, workspace=None,
               stream=None):
    """q', k' = rope_apply(q, k, (cos, sin)): q [B, T, Hq, d] and k [B, T, Hkv,
    d] (either may be None) turned by rotary tables [rows, rot/2], rot <= d,
    at positions ``pos`` int32 [B, T] (None: t). ``inverse``: the transposed
    rotation, which turns gradients of q', k' into those of q, k. ``out`` =
    (q', k') may be (q, k): in place. ``workspace``: where positions outside
    the tables are reported (swa_attn_check_status), which nothing tells
    without one. Their rows are zero in new outputs, and left as they were in
    those of ``out``."""
    if _fast is not None and stream is None and rope is not None:
        r = _fast.rope_apply(q, k, *rope, pos, interleaved, inverse, *(_NO_ROPE if out is None else out), workspace)
        if r is not None:
            return r
    x = q if q is not None else k
    if x is None or x.dim() != 4:
        raise ValueError("rope_apply: q or k [B, T, H, d] is expected")
    dt, dev = x.dtype, x.device
    lib = load(_kind("q, k", dt))
    B, T, Hq, d = x.shape
    Hkv = k.shape[2] if q is not None and k is not None else (1 if k is None else Hq)
    qo, ko = (None, None) if out is None else out
    sq, sk = (B, T, Hq, d), (B, T, Hkv, d)
    qa, ka, qoa, koa = _at("q", q, dt, sq, dev), _at("k", k, dt, sk, dev), _at("out of q", qo, dt, sq, dev), \
        _at("out of k", ko, dt, sk, dev)
    pa = _at("pos", pos, _I32, (B, T), dev)
    r = _rope_at(rope, interleaved, dev)
    ws, nws = _ws_at(workspace, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: rope_apply(q, k, rope, pos=pos, interleaved=interleaved, inverse=inverse, out=out,
                                                      workspace=workspace))
    # outputs allocated here hold nothing yet: the call is told so, or, beside
    # one of the caller's, they begin as zeros where a row may be left out
    fresh = qo is None and ko is None
    new = torch.empty_like if fresh or pos is None else torch.zeros_like
    if q is not None and qo is None:
        qo = new(q)
        qoa = qo.data_ptr()
    if k is not None and ko is None:
        ko = new(k)
        koa = ko.data_ptr()
    s = lib.swa_rope_apply(swa_params(B, T, Hq, Hkv, d, -1, 1, 0.0, 0.0, 0.0, 0), r, pa, qa, ka, qoa, koa,
                           (1 if inverse else 0) | (SWA_ROPE_NEW_OUTPUTS if fresh else 0), ws, nws, st)
    if s:
        raise SwaError(s, "swa_rope_apply")
    return qo, ko


def _cache_dims(cache):
    """n_pages, Hkv, page, d of a cache tensor (new_kv4_cache)."""
    n, Hkv, tiles, row = cache.shape if cache.dim() == 4 else (0, 0, 0, 0)
    if row not in (18 * 64, 18 * 128) or cache.dtype is not _U8 or not cache.is_contiguous():
        raise ValueError("cache: a contiguous uint8 tensor [pages, Hkv, page / 16, 18 d] is expected, d 64 or 128")
    return n, Hkv, 16 * tiles, row // 18


def new_kv4_cache(n_pages: int, page: int, Hkv: int, d: int, device):
    """A 4-bit paged cache of one layer, uint8 [n_pages, Hkv, page/16, 18 d]:
    ``page`` (a multiple of 16) tokens of keys and values to a page. Zeroed."""
    p = make_params(1, 1, Hkv, Hkv, d)
    if swa_kv4_cache_size(p, n_pages, page) == 0:
        raise SwaError(SWA_ERR_INVALID_ARG, "cache size")
    return torch.zeros(n_pages, Hkv, page // 16, 18 * d, dtype=torch.uint8, device=device)


def new_kv4_workspace(cache, B: int, Hq: int, *, max_pages: int, window: int = -1, kind: str = "bf16", stream=None):
    """A workspace of kv4_attention, initialised: 10 MB, the same for every
    batch, window and head count (the arguments are only checked), for calls
    that run one after the other. kind: "bf16" or "fp32", as q."""
    _, Hkv, page, d = _cache_dims(cache)
    n = swa_kv4_workspace_size(make_params(B, 1, Hq, Hkv, d, window), page, max_pages, kind)
    if n == 0:
        raise SwaError(SWA_ERR_INVALID_ARG, "workspace size")

    def call():
        ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
        _check(swa_kv4_workspace_init(ws, n, None, kind), "workspace init")
        return ws
    return _there(cache.device, stream, call)


def kv4_plan(lens, new_lens, table, free_pages, free_head, *, page: int, n_pages: int, n_tokens: Optional[int] = None,
             workspace=None, stream=None) -> dict:
    """The plan of a serving step, on the GPU: request b holds lens[b] tokens
    and gets new_lens[b] more (None: one each; all int32). Pages come from
    free_pages[free_head:] (free_head int32 [1]) and are written into table
    [B, max_pages] behind those it holds. Returns slot (int64), pos, row
    (int32) of each new token [n_tokens] (the sum of new_lens, known to the
    host; more is padding, slot -1), cu [B + 1], and lens and free_head
    afterwards."""
    if _fast is not None and stream is None and n_tokens is not None:
        r = _fast.kv4_plan(lens, new_lens, table, free_pages, free_head, page, n_pages, n_tokens, workspace)
        if r is not None:
            return r
    dev = lens.device
    if table.dim() != 2 or lens.dim() != 1:
        raise ValueError("lens [B] and table [B, max_pages] are expected")
    B, max_pages = table.shape
    row_b, n_free = (B,), free_pages.numel()
    la, na = _at("lens", lens, _I32, row_b, dev), _at("new_lens", new_lens, _I32, row_b, dev)
    ta, fa = _at("table", table, _I32, table.shape, dev), _at("free_pages", free_pages, _I32, (n_free,), dev)
    ha = _at("free_head", free_head, _I32, (1,), dev)
    ws, nws = _ws_at(workspace, dev)
    if n_tokens is None:
        if new_lens is not None:
            raise ValueError("n_tokens: the number of new tokens is expected with new_lens")
        n_tokens = B
    if n_tokens < 0:
        raise ValueError("n_tokens: not below 0")

    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_plan(lens, new_lens, table, free_pages, free_head, page=page, n_pages=n_pages,
                                                    n_tokens=n_tokens, workspace=workspace))
    # one buffer for all outputs: slots first, then the int32 ones, in 16-byte aligned pieces
    pad = (n_tokens + 3) // 4 * 4
    ints = torch.empty((4 * pad + 2 * B + 2,), dtype=_I32, device=dev)
    at = ints.data_ptr()
    s = load("bf16").swa_kv4_plan(n_pages, page, B, max_pages, la, na, ta, fa, n_free, ha, n_tokens, at, at + 8 * pad,
                                  at + 12 * pad, at + 16 * pad, at + 16 * pad + 4 * (B + 1), at + 16 * pad + 4 * (2 * B + 1),
                                  ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_plan")
    slot, pos, row, cu, lens_out, head = ints.split_with_sizes((2 * pad, pad, pad, B + 1, B, 1))
    slot = slot.view(_I64)
    if pad != n_tokens:
        slot, pos, row = slot[:n_tokens], pos[:n_tokens], row[:n_tokens]
    return {"slot": slot, "pos": pos, "row": row, "cu": cu, "lens": lens_out, "free_head": head}


def kv4_append(cache, k, v, slot, *, pos=None, rope=None, interleaved: bool = False, gk=None, eps: float = 1e-6,
               ve=None, tok=None, ve_gate=None, ve_scale: float = 0.5, gate_x=None, gate_w=None, workspace=None,
               stream=None) -> None:
    """Writes new keys and values k, v [B, T, Hkv, d] (as projected: not yet
    rotated, normed or mixed) into the cache at slot int64 [B, T]; -1 skips a
    token. Rotary, QK-norm gain, value embedding and gate as in
    attention_forward, with the rotation at pos int32 [B, T] (None: t). A token
    whose slot or position is out of range is skipped, which only a
    ``workspace`` tells (swa_attn_check_status)."""
    if _fast is not None and stream is None and gate_w is None:
        if _fast.kv4_append(cache, k, v, slot, pos, *(_NO_ROPE if rope is None else rope), interleaved, gk, eps, ve, tok, ve_gate, ve_scale,
                            workspace):
            return
    n_pages, Hkv, page, d = _cache_dims(cache)
    dev, dt = cache.device, k.dtype
    lib = load(_kind("k", dt))
    if k.dim() != 4:
        raise ValueError("k: [B, T, Hkv, d] is expected")
    B, T = k.shape[:2]
    rows, tokens = (B, T, Hkv, d), (B, T)
    ka, va = _at("k", k, dt, rows, dev), _at("v", v, dt, rows, dev)
    sa, pa = _at("slot", slot, _I64, tokens, dev), _at("pos", pos, _I32, tokens, dev)
    ga = _at("gk", gk, _F32, (d,), dev)
    vocab, ex, ea, ta, gta = 0, None, None, None, None
    if ve is not None:
        vocab = ve.shape[0]
        ea, ta = _at("ve", ve, dt, (vocab, Hkv * d), dev), _at("tok", tok, _I32, tokens, dev)
        gta = _at("ve_gate", ve_gate, _F32, (B, T, Hkv), dev)
        if gate_w is not None:
            if gate_w.dim() != 2:
                raise ValueError("gate_w: [Hkv, channels] is expected")
            _at("gate_w", gate_w, _F32, (Hkv, gate_w.shape[1]), dev)
            if gate_x is None or gate_x.dtype is not dt or gate_x.device != dev or gate_x.dim() != 3 \
                    or gate_x.shape[:2] != tokens or gate_x.shape[2] < gate_w.shape[1]:
                raise ValueError(f"gate_x: a {dt} tensor [B, T, channels] on {dev} is expected")
            ex = make_extras(None, gate_x, gate_w)
    r = _rope_at(rope, interleaved, dev)
    ws, nws = _ws_at(workspace, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_append(
            cache, k, v, slot, pos=pos, rope=rope, interleaved=interleaved, gk=gk, eps=eps, ve=ve, tok=tok, ve_gate=ve_gate,
            ve_scale=ve_scale, gate_x=gate_x, gate_w=gate_w, workspace=workspace))
    s = lib.swa_kv4_append(swa_params(B, T, Hkv, Hkv, d, -1, 1, 0.0, eps, ve_scale, vocab), ex,
                           swa_kv4_cache(cache.data_ptr(), n_pages, page), r, ka, va, ga, ea, ta, gta, pa, sa, ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_append")


def kv4_read(cache, slot, *, dtype=torch.bfloat16, workspace=None, stream=None):
    """k, v = kv4_read(cache, slot): the rows that slot int64 [B, T] holds, as
    ``dtype`` (bf16 or fp32) [B, T, Hkv, d]; keys are rotated and normed.
    Rows of slot -1, and of slots outside the cache (reported in
    ``workspace``), are zero."""
    if _fast is not None and stream is None and (dtype is _BF16 or dtype is _F32):
        r = _fast.kv4_read(cache, slot, dtype is _F32, workspace)
        if r is not None:
            return r
    n_pages, Hkv, page, d = _cache_dims(cache)
    dev = cache.device
    lib = load(_kind("dtype", dtype))
    if slot.dim() != 2:
        raise ValueError("slot: [B, T] is expected")
    B, T = slot.shape
    sa = _at("slot", slot, _I64, (B, T), dev)
    ws, nws = _ws_at(workspace, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_read(cache, slot, dtype=dtype, workspace=workspace))
    k = torch.empty((B, T, Hkv, d), dtype=dtype, device=dev)
    v = torch.empty_like(k)
    s = lib.swa_kv4_read(swa_params(B, T, Hkv, Hkv, d, -1, 1, 0.0, 0.0, 0.0, 0),
                         swa_kv4_cache(cache.data_ptr(), n_pages, page), sa, k.data_ptr(), v.data_ptr(), ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_read")
    return k, v


def kv4_attention(cache, q, table, lens, *, rope=None, interleaved: bool = False, gq=None, window: int = -1,
                  softmax_scale: float = 0.0, eps: float = 1e-6, workspace=None, stream=None):
    """o, lse = kv4_attention(cache, q, table, lens): attention of one token
    per request, q [B, Hq, d] (as projected), at position lens[b] - 1 over the
    request's cached keys and values (its own among them), table int32 [B,
    max_pages]. o as q; lse fp32 [B, Hq]. Rotary, gain, window and scale as in
    attention_forward. ``workspace``: from new_kv4_workspace, kept by the
    caller (one per stream), where numbers out of range are reported; None: one
    for this call, and its reports are lost."""
    if _fast is not None and stream is None:
        r = _fast.kv4_attention(cache, q, table, lens, *(_NO_ROPE if rope is None else rope), interleaved, gq, window,
                                softmax_scale, eps, workspace)
        if r is not None:
            return r
    n_pages, Hkv, page, d = _cache_dims(cache)
    dev, dt = cache.device, q.dtype
    kind = _kind("q", dt)
    if q.dim() != 3 or table.dim() != 2:
        raise ValueError("q [B, Hq, d] and table [B, max_pages] are expected")
    B, Hq = q.shape[:2]
    max_pages = table.shape[1]
    qa, ga = _at("q", q, dt, (B, Hq, d), dev), _at("gq", gq, _F32, (d,), dev)
    ta, la = _at("table", table, _I32, (B, max_pages), dev), _at("lens", lens, _I32, (B,), dev)
    r = _rope_at(rope, interleaved, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_attention(
            cache, q, table, lens, rope=rope, interleaved=interleaved, gq=gq, window=window, softmax_scale=softmax_scale,
            eps=eps, workspace=workspace))
    if workspace is None:
        workspace = new_kv4_workspace(cache, B, Hq, max_pages=max_pages, window=window, kind=kind)
    ws, nws = _ws_at(workspace, dev)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=_F32, device=dev)
    s = load(kind).swa_kv4_attn(swa_params(B, 1, Hq, Hkv, d, window, 1, softmax_scale, eps, 0.0, 0), None,
                                swa_kv4_cache(cache.data_ptr(), n_pages, page), r, qa, ga, ta, max_pages, la, o.data_ptr(),
                                lse.data_ptr(), ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_attn")
    return o, lse


# ---------------------------------------------------------------------------
# Drafted tokens, the norm and the 4-bit projections of a serving step (and the
# norm's backward). Checks, devices and streams as above.
# ---------------------------------------------------------------------------

_F8 = torch.float8_e4m3fn


def kv4_tree(parent, cu, lens, *, max_new: int, workspace=None, stream=None):
    """pos, seen = kv4_tree(parent, cu, lens): positions (int32) and visibility
    (int64 bits) of a step's drafted tokens, from parent int32 [N] (the index of
    each token's parent among its request's, -1: the context), cu int32 [B + 1]
    (rows of the requests; those in front of cu[0] and behind cu[B] are padding) and lens int32 [B]
    (cached tokens, the drafted ones among them: cu and lens of kv4_plan). At
    most ``max_new`` (up to 64) tokens a request."""
    if _fast is not None and stream is None:
        r = _fast.kv4_tree(parent, cu, lens, max_new, workspace)
        if r is not None:
            return r
    dev = parent.device
    if parent.dim() != 1 or cu.dim() != 1 or cu.numel() < 1:
        raise ValueError("parent [N] and cu [B + 1] are expected")
    N, B = parent.shape[0], cu.shape[0] - 1
    pa, ca, la = _at("parent", parent, _I32, (N,), dev), _at("cu", cu, _I32, (B + 1,), dev), _at("lens", lens, _I32, (B,), dev)
    ws, nws = _ws_at(workspace, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_tree(parent, cu, lens, max_new=max_new, workspace=workspace))
    pos = torch.empty((N,), dtype=_I32, device=dev)
    seen = torch.empty((N,), dtype=_I64, device=dev)
    s = load("bf16").swa_kv4_tree(B, N, max_new, pa, ca, la, pos.data_ptr(), seen.data_ptr(), ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_tree")
    return pos, seen


def kv4_tree_attention(cache, q, table, lens, cu, pos, seen, *, max_new: int, rope=None, interleaved: bool = False, gq=None,
                       window: int = -1, softmax_scale: float = 0.0, eps: float = 1e-6, workspace=None, stream=None):
    """o, lse = kv4_tree_attention(cache, q, table, lens, cu, pos, seen):
    attention of each request's drafted tokens, q [N, Hq, d] (as projected), over
    its context and the drafted tokens that ``seen`` shows it (kv4_tree), whose keys
    and values are in the cache already. The other arguments are those of
    kv4_attention. Rows that see nothing (padding among them) are 0, their lse
    -infinity."""
    if _fast is not None and stream is None:
        r = _fast.kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new, *(_NO_ROPE if rope is None else rope), interleaved,
                                     gq, window, softmax_scale, eps, workspace)
        if r is not None:
            return r
    n_pages, Hkv, page, d = _cache_dims(cache)
    dev, dt = cache.device, q.dtype
    kind = _kind("q", dt)
    if q.dim() != 3 or table.dim() != 2:
        raise ValueError("q [N, Hq, d] and table [B, max_pages] are expected")
    N, Hq = q.shape[:2]
    B, max_pages = table.shape
    qa, ga = _at("q", q, dt, (N, Hq, d), dev), _at("gq", gq, _F32, (d,), dev)
    ta, la = _at("table", table, _I32, (B, max_pages), dev), _at("lens", lens, _I32, (B,), dev)
    ca, pa, sa = _at("cu", cu, _I32, (B + 1,), dev), _at("pos", pos, _I32, (N,), dev), _at("seen", seen, _I64, (N,), dev)
    r = _rope_at(rope, interleaved, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_tree_attention(
            cache, q, table, lens, cu, pos, seen, max_new=max_new, rope=rope, interleaved=interleaved, gq=gq, window=window,
            softmax_scale=softmax_scale, eps=eps, workspace=workspace))
    if workspace is None:
        workspace = new_kv4_workspace(cache, B, Hq, max_pages=max_pages, window=window, kind=kind)
    ws, nws = _ws_at(workspace, dev)
    o = torch.empty_like(q)
    lse = torch.empty((N, Hq), dtype=_F32, device=dev)
    s = load(kind).swa_kv4_tree_attn(swa_params(B, 1, Hq, Hkv, d, window, 1, softmax_scale, eps, 0.0, 0), None,
                                     swa_kv4_cache(cache.data_ptr(), n_pages, page), r, N, max_new, qa, ga, ta, max_pages, la, ca,
                                     pa, sa, o.data_ptr(), lse.data_ptr(), ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_tree_attn")
    return o, lse


def kv4_move(cache, src, dst, *, workspace=None, stream=None) -> None:
    """Moves cached tokens: those of slots src int64 [B, T] (T <= 64) become those of
    dst. All of a row are read before any is written; rows must not write what
    others read or write. -1 in either skips a pair; slots outside the cache are
    skipped, which only a ``workspace`` tells."""
    if _fast is not None and stream is None and _fast.kv4_move(cache, src, dst, workspace):
        return
    n_pages, Hkv, page, d = _cache_dims(cache)
    dev = cache.device
    if src.dim() != 2:
        raise ValueError("src: [B, T] is expected")
    B, T = src.shape
    sa, da = _at("src", src, _I64, (B, T), dev), _at("dst", dst, _I64, (B, T), dev)
    ws, nws = _ws_at(workspace, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_move(cache, src, dst, workspace=workspace))
    s = load("bf16").swa_kv4_move(swa_params(B, T, Hkv, Hkv, d, -1, 1, 0.0, 0.0, 0.0, 0),
                                  swa_kv4_cache(cache.data_ptr(), n_pages, page), sa, da, ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_move")


def _rows_of(name, x):
    if x.dim() < 1:
        raise ValueError(f"{name}: [..., channels] is expected")
    C = x.shape[-1]
    return (x.numel() // C if C else 0), C


def rms_norm(x, gain=None, *, add=None, eps: float = 1e-6, fp8: bool = False, inplace: bool = False, stream=None) -> dict:
    """h = x + add, y = gain h / sqrt(mean(h^2) + eps) over the last dimension of
    x (bf16 or fp32; gain fp32 [C]). Returns y, h (x itself without an ``add``) and
    rstd fp32 [...]; with ``fp8`` y is float8_e4m3fn and scale fp32 [...] the rows'
    factors (y ~ y * scale). ``inplace``: h is written over x."""
    if _fast is not None and stream is None:
        r = _fast.rms_norm(x, gain, add, eps, fp8, inplace)
        if r is not None:
            return r
    rows, C = _rows_of("x", x)
    dt, dev = x.dtype, x.device
    lib = load(_kind("x", dt))
    xa, aa, ga = _at("x", x, dt, x.shape, dev), _at("add", add, dt, x.shape, dev), _at("gain", gain, _F32, (C,), dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: rms_norm(x, gain, add=add, eps=eps, fp8=fp8, inplace=inplace))
    h = x if add is None or inplace else torch.empty_like(x)
    y = torch.empty(x.shape, dtype=_F8 if fp8 else dt, device=dev)
    rstd = torch.empty(x.shape[:-1], dtype=_F32, device=dev)
    scale = torch.empty_like(rstd) if fp8 else None
    # (an empty tensor has no address; nothing is written then)
    ya = y.data_ptr() or 256
    s = lib.swa_rms_norm(rows, C, eps, xa, aa, ga, h.data_ptr() if add is not None else None, None if fp8 else ya, ya if fp8 else None,
                         (scale.data_ptr() or 256) if fp8 else None, rstd.data_ptr(), st)
    if s:
        raise SwaError(s, "swa_rms_norm")
    return {"y": y, "scale": scale, "h": h, "rstd": rstd}


def rms_norm_backward(h, rstd, dy, gain=None, *, dh=None, need_gain: bool = True, workspace=None, stream=None) -> dict:
    """Backward of rms_norm from its h and rstd: dx, the gradient of x and of add
    (dy's, and dh where h is used elsewhere: the residual), and dgain fp32 [C] (None
    without ``need_gain``). ``workspace``: uint8, of swa_rms_norm_workspace_size
    bytes; None: one for this call."""
    if _fast is not None and stream is None and need_gain:
        r = _fast.rms_norm_backward(h, rstd, dy, gain, dh, workspace)
        if r is not None:
            return r
    rows, C = _rows_of("h", h)
    dt, dev = h.dtype, h.device
    kind = _kind("h", dt)
    ha, da, ea = _at("h", h, dt, h.shape, dev), _at("dy", dy, dt, h.shape, dev), _at("dh", dh, dt, h.shape, dev)
    ra, ga = _at("rstd", rstd, _F32, h.shape[:-1], dev), _at("gain", gain, _F32, (C,), dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: rms_norm_backward(h, rstd, dy, gain, dh=dh, need_gain=need_gain, workspace=workspace))
    dx = torch.empty_like(h)
    dgain = torch.empty((C,), dtype=_F32, device=dev) if need_gain else None
    if workspace is None and need_gain:
        workspace = torch.empty((swa_rms_norm_workspace_size(rows, C, kind),), dtype=_U8, device=dev)
    ws, nws = _ws_at(workspace, dev)
    s = load(kind).swa_rms_norm_bwd(rows, C, ha, ra, ga, da, ea, dx.data_ptr(), dgain.data_ptr() if need_gain else None, ws, nws, st)
    if s:
        raise SwaError(s, "swa_rms_norm_bwd")
    return {"dx": dx, "dgain": dgain}


def _w4_tiles(N: int, K: int):
    return -(-N // 16), -(-K // 64), 544


def w4_pack(w, *, stream=None):
    """Weights w [N, K] (torch.nn.Linear layout, bf16 or fp32, K a multiple of 8) in 4
    bits with a bf16 step per row and 64 columns: uint8 [N / 16, K / 64, 544], both
    rounded up."""
    if w.dim() != 2:
        raise ValueError("w: [N, K] is expected")
    (N, K), dev = w.shape, w.device
    lib, wa = load(_kind("w", w.dtype)), _at("w", w, w.dtype, w.shape, w.device)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: w4_pack(w))
    w4 = torch.empty(_w4_tiles(N, K), dtype=_U8, device=dev)
    s = lib.swa_w4_pack(N, K, wa, w4.data_ptr(), st)
    if s:
        raise SwaError(s, "swa_w4_pack")
    return w4


def w4_unpack(w4, out_features: int, in_features: int, *, dtype=torch.bfloat16, stream=None):
    """The weights [out_features, in_features] that w4 holds, as ``dtype``."""
    lib, dev, N, K = load(_kind("dtype", dtype)), w4.device, out_features, in_features
    wa = _at("w4", w4, _U8, _w4_tiles(N, K), dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: w4_unpack(w4, N, K, dtype=dtype))
    w = torch.empty((N, K), dtype=dtype, device=dev)
    s = lib.swa_w4_unpack(N, K, wa, w.data_ptr(), st)
    if s:
        raise SwaError(s, "swa_w4_unpack")
    return w


def w4_linear(x, w4, *, out_features: Optional[int] = None, scale=None, add=None, dtype=None, out=None, workspace=None,
              stream=None):
    """y = x W^T (+ add) [..., out_features] for x [..., K] and weights of w4_pack
    (out_features: N; None: a multiple of 16, all that w4 holds). x is bf16 or fp32, or
    float8_e4m3fn with ``scale`` fp32 [...] (rms_norm's pair); then ``dtype`` is y's
    (bf16 by default). ``out``: y, which may be ``add``. ``workspace``: where a wait
    that ran out is reported (swa_attn_check_status)."""
    if _fast is not None and stream is None and (dtype is None or dtype is _BF16 or dtype is _F32):
        r = _fast.w4_linear(x, w4, out_features, scale, add, 0 if dtype is None else (1 if dtype is _BF16 else 2),
                            out, workspace)
        if r is not None:
            return r
    M, K = _rows_of("x", x)
    dev = x.device
    if w4.dim() != 3:
        raise ValueError("w4: uint8 [N / 16, K / 64, 544] is expected")
    N = 16 * w4.shape[0] if out_features is None else out_features
    if scale is None:
        if dtype is not None and dtype is not x.dtype:
            raise ValueError(f"dtype: that of x, {x.dtype}, is expected, got {dtype}")
        dt = x.dtype
    else:
        dt = _BF16 if dtype is None else dtype
    lib = load(_kind("dtype" if scale is not None else "x", dt))
    shape = (*x.shape[:-1], N)
    xa, wa = _at("x", x, dt if scale is None else _F8, x.shape, dev), _at("w4", w4, _U8, _w4_tiles(N, K), dev)
    sa, aa, oa = _at("scale", scale, _F32, x.shape[:-1], dev), _at("add", add, dt, shape, dev), _at("out", out, dt, shape, dev)
    ws, nws = _ws_at(workspace, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: w4_linear(x, w4, out_features=N, scale=scale, add=add, dtype=dt, out=out,
                                                     workspace=workspace))
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
        oa = out.data_ptr()
    s = lib.swa_w4_linear(M, N, K, xa, sa, wa, aa, oa, ws, nws, st)
    if s:
        raise SwaError(s, "swa_w4_linear")
    return out


def new_kv4_block_workspace(cache, n_tokens: int, C: int, Hq: int, *, kind: str = "bf16", stream=None):
    """A workspace of kv4_block for steps of up to ``n_tokens`` tokens of width C,
    initialised; the other decode calls may use it too."""
    _, Hkv, _, d = _cache_dims(cache)
    n = swa_kv4_block_workspace_size(make_params(1, 1, Hq, Hkv, d), C, n_tokens, kind)
    if n == 0:
        raise SwaError(SWA_ERR_INVALID_ARG, "workspace size")

    def call():
        ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
        _check(swa_kv4_workspace_init(ws, n, None, kind), "workspace init")
        return ws
    return _there(cache.device, stream, call)


def kv4_block(cache, x, weights, table, lens, slot, pos, *, Hq: int, cu=None, seen=None, max_new: int = 1, add=None, gain=None,
              rope=None, interleaved: bool = False, gq=None, gk=None, ve=None, tok=None, gate_w=None, ve_scale: float = 0.5,
              window: int = -1, softmax_scale: float = 0.0, eps: float = 1e-6, out=None, workspace=None, stream=None):
    """out = h + c_proj(attention(norm(h))), h = x + add: a serving step of the whole
    attention block over the 4-bit cache for the tokens x [N, C], with weights =
    (wq, wk, wv, wo), each of w4_pack. slot int64 [N], pos int32 [N], lens: as
    kv4_plan gives them. One token a request (N = B), or drafted tokens with cu, pos
    and seen of kv4_tree and ``max_new``. gain fp32 [C]: of the pre-norm; gate_w fp32
    [Hkv, C' <= 32]: the learned gate of value embeddings ve, tok [N]; the rest as in
    kv4_append and kv4_attention. ``workspace``: of new_kv4_block_workspace (None: one
    for this call, whose reports are lost)."""
    n_pages, Hkv, page, d = _cache_dims(cache)
    dev, dt = cache.device, x.dtype
    kind = _kind("x", dt)
    if x.dim() != 2 or table.dim() != 2 or len(weights) != 4:
        raise ValueError("x [N, C], table [B, max_pages] and weights (wq, wk, wv, wo) are expected")
    N, C = x.shape
    B, max_pages = table.shape
    if (cu is None) != (seen is None) or (cu is None and N != B):
        raise ValueError("cu and seen, or one token a request, are expected")
    nq, nk = Hq * d, Hkv * d
    wa = [_at(n, w, _U8, _w4_tiles(*s), dev) for n, w, s in zip(("wq", "wk", "wv", "wo"), weights, ((nq, C), (nk, C), (nk, C), (C, nq)))]
    xa, aa, oa = _at("x", x, dt, (N, C), dev), _at("add", add, dt, (N, C), dev), _at("out", out, dt, (N, C), dev)
    na, qa, ka = _at("gain", gain, _F32, (C,), dev), _at("gq", gq, _F32, (d,), dev), _at("gk", gk, _F32, (d,), dev)
    vocab, ea, ka2, ex = 0, None, None, None
    if ve is not None:
        vocab = ve.shape[0]
        ea, ka2 = _at("ve", ve, dt, (vocab, nk), dev), _at("tok", tok, _I32, (N,), dev)
        if gate_w is not None:
            if gate_w.dim() != 2:
                raise ValueError("gate_w: [Hkv, channels] is expected")
            ex = swa_extras()
            ex.gate_w, ex.gate_ch = _at("gate_w", gate_w, _F32, (Hkv, gate_w.shape[1]), dev), gate_w.shape[1]
    sa, pa = _at("slot", slot, _I64, (N,), dev), _at("pos", pos, _I32, (N,), dev)
    ta, la = _at("table", table, _I32, (B, max_pages), dev), _at("lens", lens, _I32, (B,), dev)
    ca, va = _at("cu", cu, _I32, (B + 1,), dev), _at("seen", seen, _I64, (N,), dev)
    r = _rope_at(rope, interleaved, dev)
    st = _stream_here(dev, stream)
    if st is None:
        return _there(dev, stream, lambda: kv4_block(
            cache, x, weights, table, lens, slot, pos, Hq=Hq, cu=cu, seen=seen, max_new=max_new, add=add, gain=gain, rope=rope,
            interleaved=interleaved, gq=gq, gk=gk, ve=ve, tok=tok, gate_w=gate_w, ve_scale=ve_scale, window=window,
            softmax_scale=softmax_scale, eps=eps, out=out, workspace=workspace))
    if workspace is None:
        workspace = new_kv4_block_workspace(cache, N, C, Hq, kind=kind)
    ws, nws = _ws_at(workspace, dev)
    if out is None:
        out = torch.empty_like(x)
        oa = out.data_ptr()
    s = load(kind).swa_kv4_block(swa_params(B, 1, Hq, Hkv, d, window, 1, softmax_scale, eps, ve_scale, vocab), ex,
                                 swa_kv4_cache(cache.data_ptr(), n_pages, page), r, swa_kv4_weights(C, *wa), N, max_new, xa, aa, na, qa,
                                 ka, ea, ka2, sa, pa, ca, va, ta, max_pages, la, oa, ws, nws, st)
    if s:
        raise SwaError(s, "swa_kv4_block")
    return out

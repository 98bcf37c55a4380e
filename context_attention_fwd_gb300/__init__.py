"""Ring-chunked exact attention for GB300 (sm_103a): thin Python binding.

Every computation runs in the CUDA library ``_build/libctxattn.so`` through
its C ABI (``include/ctx_attn.h``); this module only marshals torch tensors
into ``ctx_tensor_t`` descriptors, allocates outputs and workspace with torch,
and passes the current CUDA stream.  The windowed, decoding, rotary and norm
calls do that part natively (``csrc/binding.cpp``), the others with ctypes.
There is no CPU path: if the library is missing or a call fails, an exception
is raised.

Tensors are *logical* ``[B, S, H, D]`` views (``.permute(1, 0, 2, 3)`` of a
sequence-first ``[S, B, H, D]`` tensor is one); their strides tell the
library how they are stored.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math
import os
import struct
import threading
from dataclasses import dataclass

import torch

from . import build as _build

__all__ = [
    "attn_fwd", "attn_bwd", "attn_window_fwd", "attn_window_bwd", "window_workspace_size", "attn_decode",
    "decode_workspace_size", "seq_head_exchange", "exchanged_view", "workspace_size",
    "chunk_offsets", "device_status", "selftest_wait_timeout", "library_path", "load_library",
    "profile_enable", "profile_read", "launch_plan", "debug_set", "kernel_binary_version",
    "RopeTable", "rope_table", "rope_fwd", "rope_bwd", "qk_norm_rope_fwd", "qk_norm_rope_bwd",
    "CtxError", "FLAG_MATERIALIZE_PARTIALS", "FLAG_KV_ALLGATHER", "DEBUG_SKIP_ARRIVAL",
]

FLAG_MATERIALIZE_PARTIALS = 1
FLAG_KV_ALLGATHER = 2
DEBUG_SKIP_ARRIVAL = 1
LAYOUT_BSHD, LAYOUT_SBHD = 0, 1
_lock = threading.Lock()
_lib = None
_binding = None


class CtxError(RuntimeError):
    def __init__(self, code: int, what: str):
        msg = _status_text(code)
        super().__init__(f"{what}: {msg} (status {code})")
        self.code = code


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("B", ctypes.c_int64), ("S", ctypes.c_int64),
                ("H", ctypes.c_int64), ("D", ctypes.c_int64), ("stride_b", ctypes.c_int64),
                ("stride_s", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class _Rope(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("n_axes", ctypes.c_int), ("sections", ctypes.c_int * 4), ("magnitude", ctypes.c_float),
                ("positions", ctypes.c_void_p), ("pos_stride_b", ctypes.c_int64), ("pos_stride_s", ctypes.c_int64),
                ("pos_stride_axis", ctypes.c_int64), ("offset", ctypes.c_int64)]


class _Plan(ctypes.Structure):
    _fields_ = [("fwd_ctas", ctypes.c_int64), ("bwd_ctas", ctypes.c_int64), ("fwd_head_major", ctypes.c_int),
                ("bwd_head_major", ctypes.c_int), ("bwd_group_split", ctypes.c_int)]


def library_path() -> str:
    return _build.LIB


def load_library(build_if_missing: bool = True):
    """Load libctxattn.so (building it first if asked and it is missing/stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library not built: {path} (run build())")
            lib = ctypes.CDLL(path)
            P, I, F, SZ, V = ctypes.POINTER, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
            T = P(_Tensor)
            lib.ctx_attn_fwd.argtypes = [T, T, T, I, P(I), I, I, F, T, V, V, SZ, I, V]
            lib.ctx_attn_bwd.argtypes = [T, T, T, T, V, T, I, P(I), I, I, F, T, T, T, V, SZ, V]
            lib.ctx_seq_head_exchange.argtypes = [T, V, I, I, I, I, V]
            lib.ctx_attn_workspace_size.argtypes = [I, I, I, I, I, I, I]
            lib.ctx_attn_workspace_size.restype = SZ
            lib.ctx_chunk_offsets.argtypes = [I, I, P(I)]
            lib.ctx_exchange_padded_len.argtypes = [ctypes.c_int64, I, I]
            lib.ctx_exchange_padded_len.restype = ctypes.c_int64
            lib.ctx_get_device_status.argtypes = [V]
            lib.ctx_selftest_wait_timeout.argtypes = [ctypes.c_uint, V]
            lib.ctx_selftest_exp2.argtypes = [V, V, V, ctypes.c_int64, V]
            lib.ctx_profile_enable.argtypes = [I]
            lib.ctx_profile_read.argtypes = [I, P(ctypes.c_double), P(I)]
            lib.ctx_attn_launch_plan.argtypes = [I, I, I, I, I, I, P(I), I, P(_Plan)]
            lib.ctx_debug_set.argtypes = [ctypes.c_uint, ctypes.c_uint]
            lib.ctx_kernel_binary_version.argtypes = [P(I)]
            R = P(_Rope)
            lib.ctx_attn_window_fwd.argtypes = [T, T, T, I, P(I), I, I, I, I, I, F, T, V, V]
            lib.ctx_attn_window_bwd.argtypes = [T, T, T, T, V, T, I, P(I), I, I, I, I, I, F, T, T, T, V, SZ, V]
            lib.ctx_attn_window_workspace_size.argtypes = [I] * 10
            lib.ctx_attn_window_workspace_size.restype = SZ
            lib.ctx_attn_decode.argtypes = [T, T, T, V, I, I, I, F, T, V, V, SZ, V]
            lib.ctx_attn_decode_workspace_size.argtypes = [I] * 8
            lib.ctx_attn_decode_workspace_size.restype = SZ
            lib.ctx_rope_fwd.argtypes = [T, T, R, I, I, T, T, V]
            lib.ctx_rope_bwd.argtypes = [T, T, R, I, I, T, T, V]
            lib.ctx_qk_norm_rope_fwd.argtypes = [T, T, V, V, I, F, R, I, I, T, T, V]
            lib.ctx_qk_norm_rope_bwd.argtypes = [T, T, T, T, V, V, I, F, R, I, I, T, T, V, V, V, SZ, V]
            lib.ctx_qk_norm_rope_workspace_size.argtypes = [I]
            lib.ctx_qk_norm_rope_workspace_size.restype = SZ
            lib.ctx_status_string.argtypes = [I]
            lib.ctx_status_string.restype = ctypes.c_char_p
            for n in ("ctx_attn_fwd", "ctx_attn_bwd", "ctx_seq_head_exchange", "ctx_chunk_offsets",
                      "ctx_get_device_status", "ctx_selftest_wait_timeout", "ctx_profile_enable",
                      "ctx_profile_read", "ctx_selftest_exp2", "ctx_attn_launch_plan", "ctx_debug_set",
                      "ctx_kernel_binary_version", "ctx_rope_fwd", "ctx_rope_bwd", "ctx_qk_norm_rope_fwd",
                      "ctx_qk_norm_rope_bwd", "ctx_attn_window_fwd", "ctx_attn_window_bwd",
                      "ctx_attn_decode"):
                getattr(lib, n).restype = I
            _lib = lib
    return _lib


def _native():
    """The module that marshals torch tensors for the calls below (csrc/binding.cpp)."""
    global _binding
    if _binding is None:
        load_library()
        with _lock:
            if _binding is None:
                if not os.path.exists(_build.BINDING):
                    raise RuntimeError(f"binding not built: {_build.BINDING} (run build())")
                spec = importlib.util.spec_from_file_location(__name__ + "._binding", _build.BINDING)
                mod = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(mod)
                _binding = mod
    return _binding


def _done(answer, what: str):
    """The results of a native call, or the error its status code stands for."""
    if type(answer) is int:
        raise CtxError(answer, what)
    return answer


def _status_text(code: int) -> str:
    try:
        return load_library(False).ctx_status_string(code).decode()
    except Exception:  # library unavailable while formatting an error
        return "error"


def _check(rc: int, what: str):
    if rc != 0:
        raise CtxError(rc, what)


def _desc(t: torch.Tensor, name: str = "tensor", bits16: bool = False) -> _Tensor:
    """ctx_tensor_t of a logical [B,S,H,D] tensor.  The C ABI carries no
    element type (bf16 throughout), so the type is checked here; the
    exchange (bits16) only moves 16-bit elements and takes any such type."""
    if t.dim() != 4:
        raise ValueError(f"{name}: expected a logical [B,S,H,D] tensor, got {t.dim()} dims")
    if bits16 and t.element_size() != 2:
        raise ValueError(f"{name}: the exchange moves 16-bit elements, got {t.dtype}")
    if not bits16 and t.dtype != torch.bfloat16:
        raise ValueError(f"{name}: dtype must be torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    if t.stride(3) != 1:
        raise ValueError(f"{name}: the D dimension must be contiguous")
    B, S, H, D = t.shape
    return _Tensor(t.data_ptr(), B, S, H, D, t.stride(0), t.stride(1), t.stride(2))


def _check_types(named):
    """Ranks and element types of a call's [B,S,H,D] tensors."""
    for name, t in named:
        if t.dim() != 4:
            raise ValueError(f"{name}: expected a logical [B,S,H,D] tensor, got {t.dim()} dims")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name}: dtype must be torch.bfloat16, got {t.dtype}")


def _check_inputs(named, device, lse=None, lse_shape=None):
    """A call's tensors before anything is allocated or launched: ranks and
    element types, the lse buffer, then devices."""
    _check_types(named)
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != tuple(lse_shape)
                            or not lse.is_contiguous()):
        raise ValueError(f"lse: expected a contiguous float32 tensor of shape {tuple(lse_shape)}, "
                         f"got {lse.dtype} {tuple(lse.shape)}")
    for name, t in named + ([("lse", lse)] if lse is not None else []):
        if not t.is_cuda:
            raise ValueError(f"{name}: tensor must be on a CUDA device")
        if t.device != device:
            raise ValueError(f"{name}: on {t.device}, the other tensors are on {device}")


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _offsets(P, offsets):
    if offsets is None:
        return None
    off = list(offsets)
    if len(off) != P + 1:
        raise ValueError("chunk offsets need P+1 entries")
    return (ctypes.c_int * (P + 1))(*off)


def _offset_bytes(P, offsets):
    return None if offsets is None else bytes(_offsets(P, offsets))


def _like_layout(t: torch.Tensor, H: int) -> torch.Tensor:
    """An empty bf16 [B,S,H,D] tensor stored in the same order as t."""
    B, S, _, D = t.shape
    if t.stride(0) >= t.stride(1):  # [B,S,H,D] storage
        return torch.empty(B, S, H, D, dtype=torch.bfloat16, device=t.device)
    return torch.empty(S, B, H, D, dtype=torch.bfloat16, device=t.device).permute(1, 0, 2, 3)


def launch_plan(B, S, Hq, Hkv, D, P, chunk_offsets=None, causal=False) -> dict:
    """How the attention calls of these sizes will be launched (host only):
    CTA counts, launch order (heads first or not) and the D=256 backward's
    GQA group split."""
    plan = _Plan()
    _check(load_library().ctx_attn_launch_plan(B, S, Hq, Hkv, D, P, _offsets(P, chunk_offsets), int(causal),
                                               ctypes.byref(plan)), "ctx_attn_launch_plan")
    return {name: getattr(plan, name) for name, _ in _Plan._fields_}


def workspace_size(B, S, Hq, Hkv, D, P, flags=0) -> int:
    return int(load_library().ctx_attn_workspace_size(B, S, Hq, Hkv, D, P, flags))


def chunk_offsets(S: int, P: int):
    """array_split chunk offsets computed by the library's host code."""
    arr = (ctypes.c_int * (P + 1))()
    _check(load_library().ctx_chunk_offsets(S, P, arr), "ctx_chunk_offsets")
    return list(arr)


def _workspace(nbytes: int, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def attn_fwd(q, k, v, P, chunk_offsets=None, causal=False, scale=None, out=None, lse=None,
             flags=0, workspace=None):
    """Ring-chunked attention forward -> (out bf16 [B,S,Hq,D] like q, lse fp32 [B,Hq,S])."""
    lib = load_library()
    named = [("q", q), ("k", k), ("v", v)] + ([("out", out)] if out is not None else [])
    _check_types(named)
    B, S, Hq, D = q.shape
    _check_inputs(named, q.device, lse, (B, Hq, S))
    out = _like_layout(q, Hq) if out is None else out
    lse = torch.empty(B, Hq, S, dtype=torch.float32, device=q.device) if lse is None else lse
    nbytes = (lib.ctx_attn_workspace_size(B, S, Hq, k.shape[2], D, P, flags)
              if flags & FLAG_MATERIALIZE_PARTIALS else 0)
    ws, wsb = _workspace(nbytes, q.device, workspace)
    rc = lib.ctx_attn_fwd(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)), P,
                          _offsets(P, chunk_offsets), LAYOUT_BSHD, int(causal),
                          float(scale) if scale else 0.0, ctypes.byref(_desc(out)),
                          ctypes.c_void_p(lse.data_ptr()),
                          ctypes.c_void_p(ws.data_ptr() if ws is not None else 0), wsb, flags,
                          _stream(q))
    _check(rc, "ctx_attn_fwd")
    return out, lse


def attn_bwd(q, k, v, out, lse, dout, P, chunk_offsets=None, causal=False, scale=None,
             dq=None, dk=None, dv=None, workspace=None):
    """Ring-chunked attention backward -> (dq, dk, dv) bf16, stored like q / k."""
    lib = load_library()
    named = [("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)]
    named += [(n, t) for n, t in (("dq", dq), ("dk", dk), ("dv", dv)) if t is not None]
    _check_types(named)
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    _check_inputs(named, q.device, lse, (B, Hq, S))
    dq = _like_layout(q, Hq) if dq is None else dq
    dk = _like_layout(k, Hkv) if dk is None else dk
    dv = _like_layout(k, Hkv) if dv is None else dv
    nbytes = lib.ctx_attn_workspace_size(B, S, Hq, Hkv, D, P, 0)
    ws, wsb = _workspace(nbytes, q.device, workspace)
    rc = lib.ctx_attn_bwd(ctypes.byref(_desc(q)), ctypes.byref(_desc(k)), ctypes.byref(_desc(v)),
                          ctypes.byref(_desc(out)), ctypes.c_void_p(lse.data_ptr()),
                          ctypes.byref(_desc(dout)), P, _offsets(P, chunk_offsets), LAYOUT_BSHD,
                          int(causal), float(scale) if scale else 0.0, ctypes.byref(_desc(dq)),
                          ctypes.byref(_desc(dk)), ctypes.byref(_desc(dv)),
                          ctypes.c_void_p(ws.data_ptr()), wsb, _stream(q))
    _check(rc, "ctx_attn_bwd")
    return dq, dk, dv


def _window(window, sinks):
    """(left, right, sinks) of a call: an int is both sides, -1 unlimited."""
    left, right = (window, window) if isinstance(window, int) else window
    if left < -1 or right < -1 or sinks < 0:
        raise ValueError(f"window sides must be >= -1 and sinks >= 0, got {window}, {sinks}")
    big = (1 << 31) - 1
    return min(int(left), big), min(int(right), big), min(int(sinks), big)


def window_workspace_size(B, S, Hq, Hkv, D, P, window, sinks=0, causal=False) -> int:
    """Bytes of device workspace ``attn_window_bwd`` needs for these sizes."""
    return int(load_library().ctx_attn_window_workspace_size(B, S, Hq, Hkv, D, P, int(causal), *_window(window, sinks)))


def attn_window_fwd(q, k, v, P, window, sinks=0, chunk_offsets=None, causal=False, scale=None, out=None, lse=None):
    """Attention forward under a sliding window with sink tokens -> (out, lse)
    as ``attn_fwd`` returns them.

    ``window`` (left, right), or one int for both: query i sees keys i - left
    .. i + right (-1: unlimited; causal: nothing after i), and the first
    ``sinks`` keys of the sequence.  A causal window of W tokens, the query's
    own among them, is (W - 1, 0)."""
    left, right, sinks = _window(window, sinks)
    return _done(_native().window_fwd(q, k, v, P, _offset_bytes(P, chunk_offsets), bool(causal), left, right, sinks,
                                      scale or 0.0, out, lse), "ctx_attn_window_fwd")


def attn_window_bwd(q, k, v, out, lse, dout, P, window, sinks=0, chunk_offsets=None, causal=False, scale=None,
                    dq=None, dk=None, dv=None, workspace=None):
    """Gradients through ``attn_window_fwd`` -> (dq, dk, dv) bf16, stored like q / k."""
    left, right, sinks = _window(window, sinks)
    return _done(_native().window_bwd(q, k, v, out, lse, dout, P, _offset_bytes(P, chunk_offsets), bool(causal), left,
                                      right, sinks, scale or 0.0, dq, dk, dv, workspace), "ctx_attn_window_bwd")


def decode_workspace_size(B, T, Hq, Hkv, D, capacity, window=-1, sinks=0) -> int:
    """Bytes of device workspace ``attn_decode`` needs for these sizes (may be 0)."""
    left, _, sinks = _window((window, 0), sinks)
    return int(load_library().ctx_attn_decode_workspace_size(B, T, Hq, Hkv, D, capacity, left, sinks))


def attn_decode(q, k, v, lengths=None, window=-1, sinks=0, scale=None, out=None, lse=None, workspace=None):
    """Attention of the newest T tokens of each sequence over its cache ->
    (out bf16 [B,T,Hq,D] like q, lse fp32 [B,Hq,T]).

    q [B,T,Hq,D]; k, v [B,capacity,Hkv,D] views of the cache, the new tokens'
    rows included; ``lengths`` int32 [B] on the device (None: the caches are
    full).  Query t is at position length - T + t; it sees the keys up to
    itself, of those the last ``window`` before it (-1: all) and the first
    ``sinks``.  A query before its sequence's start gives 0 and -inf."""
    left, _, sinks = _window((window, 0), sinks)
    return _done(_native().decode(q, k, v, lengths, left, sinks, scale or 0.0, out, lse, workspace), "ctx_attn_decode")


def exchanged_shape(B, S, H, D, ring, ulysses, layout):
    Sp = int(load_library().ctx_exchange_padded_len(S, ring, ulysses))
    if layout == "bshd":
        return (ulysses, B, Sp, H // ulysses, D)
    return (ulysses, Sp, B, H // ulysses, D)


def seq_head_exchange(x, ring, ulysses, direction, layout, y=None, S=None, B=None, H=None):
    """Ulysses exchange through the library.

    direction 0: x is a logical [B,S,H,D] view stored in `layout` order;
    returns y (dense, ``exchanged_shape``).  direction 1: x is y; returns the
    logical [B,S,H,D] tensor stored in `layout` order (S, B, H required)."""
    lib = load_library()
    lay = LAYOUT_BSHD if layout == "bshd" else LAYOUT_SBHD
    if direction == 0:
        B_, S_, H_, D = x.shape
        y = torch.empty(exchanged_shape(B_, S_, H_, D, ring, ulysses, layout), dtype=x.dtype,
                        device=x.device) if y is None else y
        rc = lib.ctx_seq_head_exchange(ctypes.byref(_desc(x, "x", bits16=True)), ctypes.c_void_p(y.data_ptr()),
                                       ring, ulysses, 0, lay, _stream(x))
        _check(rc, "ctx_seq_head_exchange")
        return y
    D = x.shape[-1]
    if y is None:
        if layout == "bshd":
            y = torch.empty(B, S, H, D, dtype=x.dtype, device=x.device)
        else:
            y = torch.empty(S, B, H, D, dtype=x.dtype, device=x.device).permute(1, 0, 2, 3)
    if not x.is_contiguous():
        raise ValueError("the exchanged buffer must be dense")
    rc = lib.ctx_seq_head_exchange(ctypes.byref(_desc(y, "y", bits16=True)), ctypes.c_void_p(x.data_ptr()),
                                   ring, ulysses, 1, lay, _stream(x))
    _check(rc, "ctx_seq_head_exchange")
    return y


def exchanged_view(y, S, layout):
    """Logical [U*B, S, H/U, D] view of an exchanged [U,B,Sp,H/U,D] buffer
    (layout "bshd"): every head group's whole sequence, as the attention
    calls consume it.  Pad rows past S are not part of the view."""
    if layout != "bshd":
        raise ValueError("the batched view exists for [B,S,H,D] storage; use y[u] per group")
    U, B, Sp, Hu, D = y.shape
    return y.view(U * B, Sp, Hu, D)[:, :S]


# ---------------------------------------------------------------- rotary positions, query/key norms
_PACK_ROPE = struct.Struct("P3i4ifP4q").pack  # ctx_rope_t in the C compiler's layout


@dataclass(frozen=True)
class RopeTable:
    """Frequencies of a rotary embedding, laid out once (``rope_table``)."""
    turns: torch.Tensor  # int64 [rot_dim / 2]: turns per position as a fraction of 2^64
    rot_dim: int
    interleaved: bool
    sections: tuple      # pairs per position axis
    magnitude: float

    def __post_init__(self):
        if (self.rot_dim < 2 or self.rot_dim % 2 or self.turns.dtype != torch.int64
                or tuple(self.turns.shape) != (self.rot_dim // 2,) or not self.turns.is_contiguous()
                or not 1 <= len(self.sections) <= 4 or sum(self.sections) != self.rot_dim // 2):
            raise ValueError("turns: one contiguous int64 per pair; sections: up to four counts of pairs that sum to them")

    @functools.cached_property
    def _head(self):
        """ctx_rope_t without positions, as bytes."""
        return _PACK_ROPE(self.turns.data_ptr(), self.rot_dim, int(self.interleaved), len(self.sections),
                          *self.sections, *[0] * (4 - len(self.sections)), self.magnitude, 0, 0, 0, 0, 0)


_NO_TABLE = (None, None)


def _table(table):
    return _NO_TABLE if table is None else (table._head, table.turns)


def rope_table(rot_dim, theta=10000.0, interleaved=False, sections=None, scaling="none", factor=1.0,
               original_len=None, beta_fast=32.0, beta_slow=1.0, magnitude=None, inv_freq=None,
               device=None) -> RopeTable:
    """The frequency table that the rotary calls take.

    Pair i of the first ``rot_dim`` elements turns by theta^(-2 i / rot_dim)
    radians per position.  ``interleaved``: pairs are neighbours (2 i, 2 i + 1)
    instead of (i, i + rot_dim / 2).  ``sections`` gives every position axis
    its own run of pairs with its own frequencies, theta^(-2 i / (2 n)) for a
    section of n pairs; positions then carry one value per axis.

    ``scaling`` stretches the context by ``factor``: "linear" divides every
    frequency by it; "ntk" raises theta to theta * factor^(d / (d - 2));
    "yarn" (Peng et al. 2023, "YaRN: Efficient Context Window Extension of
    Large Language Models") divides by it the frequencies that turn less than
    ``beta_slow`` times over ``original_len`` positions, keeps those that turn
    more than ``beta_fast`` times, blends linearly between, and multiplies the
    rotated part by 0.1 ln(factor) + 1.  ``magnitude`` overrides that
    multiplier; ``inv_freq`` (radians per position, one per pair) overrides
    the frequencies."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim: expected an even number >= 2, got {rot_dim}")
    secs = (rot_dim // 2,) if sections is None else tuple(int(n) for n in sections)
    if not 1 <= len(secs) <= 4 or min(secs) < 1 or sum(secs) != rot_dim // 2:
        raise ValueError(f"sections: 1 to 4 positive counts that sum to rot_dim / 2 = {rot_dim // 2}, got {secs}")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"scaling: {scaling!r} is none of 'none', 'linear', 'ntk', 'yarn'")
    if not (theta > 1.0 and math.isfinite(theta)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError(f"theta must exceed 1 and factor be at least 1, got {theta}, {factor}")
    if scaling == "yarn" and not original_len:
        raise ValueError("scaling='yarn' needs original_len")
    if inv_freq is not None:
        freq = [float(w) for w in inv_freq]
        if len(freq) != rot_dim // 2:
            raise ValueError(f"inv_freq: expected {rot_dim // 2} values, got {len(freq)}")
    else:
        freq = []
        for n in secs:
            d, base = 2 * n, float(theta)
            if scaling == "ntk":
                if d <= 2:
                    raise ValueError("scaling='ntk' needs sections of more than one pair")
                base *= factor ** (d / (d - 2.0))
            w = [base ** (-2.0 * i / d) for i in range(n)]
            if scaling == "linear":
                w = [x / factor for x in w]
            elif scaling == "yarn":
                pair = lambda turns: d * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
                lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), d - 1)
                for i in range(n):
                    slow = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                    w[i] = w[i] / factor * slow + w[i] * (1.0 - slow)
            freq += w
    if any(not 0.0 <= w < 2 * math.pi for w in freq):
        raise ValueError("frequencies must lie in [0, 2 pi) radians per position")
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1.0 else 1.0
    fixed = [int(w / (2 * math.pi) * 2.0 ** 64) for w in freq]
    turns = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in fixed], dtype=torch.int64)
    return RopeTable(turns.to("cuda" if device is None else device), int(rot_dim), bool(interleaved), secs,
                     float(magnitude))


def rope_fwd(q, k, table, positions=None, offset=0, q_out=None, k_out=None):
    """Rotary positions -> (q_out, k_out), stored like q and k (k may be None).

    q [B,S,Hq,D], k [B,S,Hk,D]: bf16, fp16 or fp32.  ``positions``: int64 [S]
    or [B,S] ([S,axes] or [B,S,axes] for a table with several axes); without
    it token s of every sequence is at ``offset + s``.  q_out / k_out may be
    q / k."""
    return _done(_native().rotate(0, *_table(table), q, k, positions, offset, q_out, k_out), "ctx_rope_fwd")


def rope_bwd(dq_out, dk_out, table, positions=None, offset=0, dq=None, dk=None):
    """Gradients through ``rope_fwd`` -> (dq, dk): the transposed rotation."""
    return _done(_native().rotate(1, *_table(table), dq_out, dk_out, positions, offset, dq, dk), "ctx_rope_bwd")


def qk_norm_rope_fwd(q, k, wq, wk, table, positions=None, offset=0, eps=1e-6, q_out=None, k_out=None):
    """Per-head RMS norm of q and k, times their weights, then the rotation, in
    one pass -> (q_out, k_out).

    wq, wk: [D] weights or None (ones); table None: the norm alone; the other
    arguments as in ``rope_fwd``."""
    return _done(_native().norm_fwd(*_table(table), q, k, wq, wk, positions, offset, eps, q_out, k_out),
                 "ctx_qk_norm_rope_fwd")


def qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, table, positions=None, offset=0, eps=1e-6, dq=None, dk=None,
                     dwq=None, dwk=None, workspace=None):
    """Gradients through ``qk_norm_rope_fwd`` -> (dq, dk, dwq, dwk).

    q, k are the forward's inputs; nothing else is saved.  dwq, dwk: fp32 [D]
    (None for a weight that is None), summed in a fixed order."""
    return _done(_native().norm_bwd(*_table(table), dq_out, dk_out, q, k, wq, wk, positions, offset, eps, dq, dk, dwq,
                                    dwk, workspace), "ctx_qk_norm_rope_bwd")


def device_status(stream=None) -> int:
    """Synchronise and read/clear the device status word (0 = ok, 5 = a wait timed out)."""
    s = torch.cuda.current_stream().cuda_stream if stream is None else stream
    return int(load_library().ctx_get_device_status(ctypes.c_void_p(s)))


def profile_enable(on: bool = True):
    """Start (clearing earlier records) or stop per-launch event timing of the
    attention kernels inside the library."""
    _check(load_library().ctx_profile_enable(int(on)), "ctx_profile_enable")


def profile_read(kernel: str):
    """(total device ms, launches) of the 'fwd' or 'bwd' attention kernel since profile_enable."""
    ms, n = ctypes.c_double(), ctypes.c_int()
    _check(load_library().ctx_profile_read(0 if kernel == "fwd" else 1, ctypes.byref(ms), ctypes.byref(n)),
           "ctx_profile_read")
    return ms.value, n.value


def selftest_exp2(x: torch.Tensor):
    """(polynomial 2^x, SFU 2^x) for a CUDA fp32 tensor x, as the kernels compute them."""
    x = x.contiguous()
    yp, ys = torch.empty_like(x), torch.empty_like(x)
    _check(load_library().ctx_selftest_exp2(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(yp.data_ptr()),
                                            ctypes.c_void_p(ys.data_ptr()), x.numel(), _stream(x)),
           "ctx_selftest_exp2")
    return yp, ys


def selftest_wait_timeout(timeout_us: int = 20000):
    s = torch.cuda.current_stream().cuda_stream
    _check(load_library().ctx_selftest_wait_timeout(timeout_us, ctypes.c_void_p(s)),
           "ctx_selftest_wait_timeout")


def debug_set(flags: int = 0, wait_limit_ms: int = 0):
    """Test-only switches of the library (``ctx_debug_set``): DEBUG_SKIP_ARRIVAL
    makes every attention kernel's producer leave out one load step so that a
    bounded device wait runs out; wait_limit_ms overrides the wait limit
    (0 = default).  ``debug_set()`` restores normal operation."""
    _check(load_library().ctx_debug_set(flags, wait_limit_ms), "ctx_debug_set")


def kernel_binary_version() -> int:
    """cudaFuncAttributes.binaryVersion of the attention kernels on the current device (103 = sm_103a)."""
    v = ctypes.c_int()
    _check(load_library().ctx_kernel_binary_version(ctypes.byref(v)), "ctx_kernel_binary_version")
    return v.value

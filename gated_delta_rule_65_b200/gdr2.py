"""Thin ctypes binding of libgdr2.so (the C ABI declared in include/gdr2.h).

Argument marshalling only: every computation happens in the library's CUDA kernels. PyTorch is used
to hold device memory and to name the current CUDA stream. If the library cannot be loaded the
calls raise; there is no fallback of any kind.

Calls go to the current stream, or to the one given as ``stream`` (a torch stream or a cudaStream_t as an
int). Outputs and workspaces that are not given are allocated as that stream's; inputs made on another
stream have to be ready for it, and outputs are waited for, as with any work on two streams.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

import torch

from . import build as _build

GDR2_F32, GDR2_BF16 = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_RANGE, ERR_BOUNDS = range(8)

EXPORTED = ("gdr2_version", "gdr2_status_string", "gdr2_check", "gdr2_workspace_bytes", "gdr2_chunk_fwd",
            "gdr2_chunk_bwd", "gdr2_decode_step", "gdr2_chunk_fwd_noalloc", "gdr2_profile_enable",
            "gdr2_profile_collect", "gdr2_chunk_fwd_train", "gdr2_chunk_bwd_saved", "gdr2_workspace_bytes_varlen",
            "gdr2_chunk_fwd_varlen", "gdr2_chunk_fwd_train_varlen", "gdr2_chunk_bwd_varlen",
            "gdr2_chunk_bwd_saved_varlen", "gdr2_gate_prologue_workspace_bytes", "gdr2_gate_prologue_fwd",
            "gdr2_gate_prologue_bwd", "gdr2_workspace_bytes_gva", "gdr2_chunk_fwd_gva", "gdr2_chunk_fwd_train_gva",
            "gdr2_chunk_bwd_gva", "gdr2_chunk_bwd_saved_gva", "gdr2_workspace_bytes_varlen_gva",
            "gdr2_chunk_fwd_varlen_gva", "gdr2_chunk_fwd_train_varlen_gva", "gdr2_chunk_bwd_varlen_gva",
            "gdr2_chunk_bwd_saved_varlen_gva", "gdr2_set_chunk_path", "gdr2_get_chunk_path", "gdr2_rope_freqs",
            "gdr2_attn_prologue_fwd", "gdr2_attn_prologue_workspace_bytes", "gdr2_attn_prologue_bwd",
            "gdr2_attn_prologue_cache", "gdr2_attn_decode_workspace_bytes", "gdr2_attn_decode",
            "gdr2_kv_workspace_bytes", "gdr2_kv_reserve", "gdr2_kv_fork", "gdr2_kv_compact", "gdr2_attn_call")

_lib = None
_lock = threading.Lock()
_VP = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
_F = ctypes.c_float
_D = ctypes.c_double


class GDR2Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {status_string(status)}")


def lib(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libgdr2.so from the package directory (building it first when missing or stale). With the
    environment variable GDR2_DEBUG_BUILD=1 the process loads libgdr2_debug.so instead: the same kernels with
    the index checks of -DGDR2_DEBUG, reported by check() as ERR_BOUNDS."""
    global _lib
    with _lock:
        if _lib is None:
            debug = os.environ.get("GDR2_DEBUG_BUILD") == "1"
            path = _build.DEBUG_LIB if debug else _build.LIB
            if build_if_missing:
                path = _build.build_debug() if debug else _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libgdr2.so not found at {path}; run gated_delta_rule_65_b200.build")
            L = ctypes.CDLL(path)
            L.gdr2_version.restype = _I
            L.gdr2_version.argtypes = []
            L.gdr2_status_string.restype = ctypes.c_char_p
            L.gdr2_status_string.argtypes = [_I]
            L.gdr2_check.restype = _I
            L.gdr2_check.argtypes = [_VP]
            L.gdr2_workspace_bytes.restype = ctypes.c_size_t
            L.gdr2_workspace_bytes.argtypes = [_I] * 7
            L.gdr2_set_chunk_path.restype = _I
            L.gdr2_set_chunk_path.argtypes = [_I]
            L.gdr2_get_chunk_path.restype = _I
            L.gdr2_get_chunk_path.argtypes = []
            L.gdr2_chunk_fwd.restype = _I
            L.gdr2_chunk_fwd.argtypes = [_VP] * 9 + [_I] * 6 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_chunk_bwd.restype = _I
            L.gdr2_chunk_bwd.argtypes = [_VP] * 16 + [_I] * 6 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_chunk_fwd_train.restype = _I
            L.gdr2_chunk_fwd_train.argtypes = [_VP] * 9 + [_I] * 6 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_chunk_bwd_saved.restype = _I
            L.gdr2_chunk_bwd_saved.argtypes = [_VP] * 16 + [_I] * 6 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_workspace_bytes_varlen.restype = ctypes.c_size_t
            L.gdr2_workspace_bytes_varlen.argtypes = [_I] * 7
            for fn in (L.gdr2_chunk_fwd_varlen, L.gdr2_chunk_fwd_train_varlen):
                fn.restype = _I
                fn.argtypes = [_VP] * 10 + [_I] * 6 + [_VP, ctypes.c_size_t, _VP]
            for fn in (L.gdr2_chunk_bwd_varlen, L.gdr2_chunk_bwd_saved_varlen):
                fn.restype = _I
                fn.argtypes = [_VP] * 17 + [_I] * 6 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_workspace_bytes_varlen_gva.restype = ctypes.c_size_t
            L.gdr2_workspace_bytes_varlen_gva.argtypes = [_I] * 8
            for fn in (L.gdr2_chunk_fwd_varlen_gva, L.gdr2_chunk_fwd_train_varlen_gva):
                fn.restype = _I
                fn.argtypes = [_VP] * 10 + [_I] * 7 + [_VP, ctypes.c_size_t, _VP]
            for fn in (L.gdr2_chunk_bwd_varlen_gva, L.gdr2_chunk_bwd_saved_varlen_gva):
                fn.restype = _I
                fn.argtypes = [_VP] * 17 + [_I] * 7 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_workspace_bytes_gva.restype = ctypes.c_size_t
            L.gdr2_workspace_bytes_gva.argtypes = [_I] * 8
            for fn in (L.gdr2_chunk_fwd_gva, L.gdr2_chunk_fwd_train_gva):
                fn.restype = _I
                fn.argtypes = [_VP] * 9 + [_I] * 7 + [_VP, ctypes.c_size_t, _VP]
            for fn in (L.gdr2_chunk_bwd_gva, L.gdr2_chunk_bwd_saved_gva):
                fn.restype = _I
                fn.argtypes = [_VP] * 16 + [_I] * 7 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_gate_prologue_workspace_bytes.restype = ctypes.c_size_t
            L.gdr2_gate_prologue_workspace_bytes.argtypes = [_I] * 6
            L.gdr2_gate_prologue_fwd.restype = _I
            L.gdr2_gate_prologue_fwd.argtypes = [_VP] * 7 + [_I] + [_VP] * 5 + [_I] * 6 + [_VP]
            L.gdr2_gate_prologue_bwd.restype = _I
            L.gdr2_gate_prologue_bwd.argtypes = ([_VP] * 7 + [_I] + [_VP] * 12 + [_I] * 6 +
                                                 [_VP, ctypes.c_size_t, _VP])
            L.gdr2_decode_step.restype = _I
            L.gdr2_decode_step.argtypes = [_VP] * 8 + [_I] * 5 + [_VP]
            L.gdr2_chunk_fwd_noalloc.restype = _I
            L.gdr2_chunk_fwd_noalloc.argtypes = [_VP] * 9 + [_I] * 6 + [_VP]
            L.gdr2_rope_freqs.restype = _I
            L.gdr2_rope_freqs.argtypes = [_VP, _VP, _I, _D, _I, _D, _D, _D, _D]
            L.gdr2_attn_prologue_fwd.restype = _I
            L.gdr2_attn_prologue_fwd.argtypes = ([_VP] * 4 + [_I, _F, _VP, _VP, _F, _I, _I, _VP, _VP] + [_I] * 5 +
                                                 [_LL] * 2 + [_VP])
            L.gdr2_attn_prologue_workspace_bytes.restype = ctypes.c_size_t
            L.gdr2_attn_prologue_workspace_bytes.argtypes = [_I]
            L.gdr2_attn_prologue_bwd.restype = _I
            L.gdr2_attn_prologue_bwd.argtypes = ([_VP] * 4 + [_I, _F, _VP, _VP, _F, _I, _I] + [_VP] * 6 + [_I] * 5 +
                                                 [_LL] * 4 + [_VP, ctypes.c_size_t, _VP])
            L.gdr2_attn_prologue_cache.restype = _I
            L.gdr2_attn_prologue_cache.argtypes = ([_VP] * 5 + [_I, _F, _VP, _VP, _VP, _F, _I, _I] + [_VP] * 4 +
                                                   [_I] * 9 + [_LL] * 3 + [_VP])
            L.gdr2_attn_decode_workspace_bytes.restype = ctypes.c_size_t
            L.gdr2_attn_decode_workspace_bytes.argtypes = [_I] * 8
            L.gdr2_attn_decode.restype = _I
            L.gdr2_attn_decode.argtypes = ([_VP] * 6 + [_F, _I, _VP, _VP] + [_I] * 9 + [_VP, ctypes.c_size_t, _VP])
            L.gdr2_kv_workspace_bytes.restype = ctypes.c_size_t
            L.gdr2_kv_workspace_bytes.argtypes = [_I] * 3
            L.gdr2_kv_reserve.restype = _I
            L.gdr2_kv_reserve.argtypes = [_VP] * 7 + [_I] * 5 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_kv_fork.restype = _I
            L.gdr2_kv_fork.argtypes = [_VP] * 10 + [_I] * 7 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_kv_compact.restype = _I
            L.gdr2_kv_compact.argtypes = [_VP] * 7 + [_I] * 7 + [_VP, ctypes.c_size_t, _VP]
            L.gdr2_attn_call.restype = _I
            L.gdr2_attn_call.argtypes = [_I, ctypes.c_char_p, ctypes.c_size_t]
            L.gdr2_profile_enable.restype = _I
            L.gdr2_profile_enable.argtypes = [_I]
            L.gdr2_profile_collect.restype = _I
            L.gdr2_profile_collect.argtypes = [ctypes.c_char_p, _I, ctypes.POINTER(_I),
                                               ctypes.POINTER(ctypes.c_double), _I, ctypes.POINTER(_I)]
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().gdr2_status_string(int(status)).decode()


def check(stream=None) -> int:
    """gdr2_check: synchronise ``stream`` (default: the current stream), then read and clear the device
    status words. Returns OK, ERR_TIMEOUT (a bounded wait expired), ERR_RANGE (a chunk's cumulative
    log-decay left [-160, 160] on the tensor-core path, [-80, 80] on the fp32 path, or an fp16 operand of the
    per-chain path passed 65504), ERR_BOUNDS (debug build only: a kernel index check failed) or ERR_CUDA; the
    outputs of the calls since the last check are valid only with OK."""
    return int(lib().gdr2_check(_stream(stream)))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDR2_F32
    if t.dtype == torch.bfloat16:
        return GDR2_BF16
    raise TypeError(f"unsupported operand dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gdr2: tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("gdr2: tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on(stream, call, args):
    """call(**args) with `stream`, given explicitly, as the current one, so that the outputs and the workspace that the
    call makes come from that stream's memory. (Out of the memory of the caller's current stream they could be what work
    still queued there writes, which `stream` does not wait for.) The results are kept for the caller's stream too, which
    may use them once it has waited."""
    del args["stream"]
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle)  # 1: the runtime's name for the legacy stream
    here = torch.cuda.current_stream()
    if stream == here:
        return call(**args)
    if stream.device != here.device:
        raise ValueError(f"gdr2: the stream is on {stream.device}, which is not the current CUDA device")
    with torch.cuda.stream(stream):
        out = call(**args)
    for t in out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,):
        if t is not None:
            t.record_stream(here)
    return out


def _check(fn, st):
    if st != OK:
        raise GDR2Error(fn, st)


PATH_AUTO, PATH_CHAIN, PATH_SPLIT = 0, 1, 2


def set_chunk_path(path: int) -> None:
    """gdr2_set_chunk_path: 0 automatic, 1 per-chain fused kernels, 2 chunk-parallel kernels (process-wide)."""
    _check("gdr2_set_chunk_path", lib().gdr2_set_chunk_path(int(path)))


def get_chunk_path() -> int:
    return int(lib().gdr2_get_chunk_path())


def workspace_bytes(B, T, H, dk, dv, dtype_code, for_bwd) -> int:
    return int(lib().gdr2_workspace_bytes(B, T, H, dk, dv, dtype_code, int(for_bwd)))


def alloc_workspace(B, T, H, dk, dv, dtype_code, for_bwd, device=None) -> torch.Tensor:
    n = workspace_bytes(B, T, H, dk, dv, dtype_code, for_bwd)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def chunk_fwd(q, k, v, log_alpha, b, w, initial_state=None, *, output_final_state=True,
              o=None, final_state=None, workspace=None, stream=None, train=False):
    """gdr2_chunk_fwd, or gdr2_chunk_fwd_train when train=True (then `workspace` must be the
    backward-sized buffer that gdr2_chunk_bwd_saved will read). Returns (o, final_state or None)."""
    if stream is not None:
        return _on(stream, chunk_fwd, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if not output_final_state:
        final_state = None
    if workspace is None:
        if train:
            raise ValueError("train=True needs the workspace that the backward will read")
        workspace = alloc_workspace(B, T, H, dk, dv, dt, 0, q.device)
    fn = lib().gdr2_chunk_fwd_train if train else lib().gdr2_chunk_fwd
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(initial_state),
                              _ptr(o), _ptr(final_state), B, T, H, dk, dv, dt, _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdr2_chunk_fwd_train" if train else "gdr2_chunk_fwd", st)
    return o, final_state


def chunk_fwd_noalloc(q, k, v, log_alpha, b, w, initial_state=None, *, output_final_state=True,
                      o=None, final_state=None, stream=None):
    """gdr2_chunk_fwd_noalloc: the forward with the library's fixed scratch instead of a workspace,
    for callers that cannot allocate device memory (the outputs here are still allocated by torch
    when not given). Returns (o, final_state or None)."""
    if stream is not None:
        return _on(stream, chunk_fwd_noalloc, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if not output_final_state:
        final_state = None
    st = lib().gdr2_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                      _ptr(initial_state), _ptr(o), _ptr(final_state), B, T, H, dk, dv,
                                      _dtype_code(q), _stream(stream))
    _check("gdr2_chunk_fwd_noalloc", st)
    return o, final_state


def chunk_bwd(q, k, v, log_alpha, b, w, initial_state=None, d_o=None, d_final_state=None, *,
              want_d_initial_state=True, out=None, workspace=None, stream=None, saved=False):
    """gdr2_chunk_bwd, or gdr2_chunk_bwd_saved when saved=True (then `workspace` is the buffer a
    chunk_fwd(..., train=True) call with the same inputs filled). Returns a dict dq, dk, dv,
    dlog_alpha, db, dw, dS0 (dS0 None if not wanted)."""
    if stream is not None:
        return _on(stream, chunk_bwd, locals())
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    if out is None:
        out = {n: torch.empty_like(q) for n in ("dq", "dk", "db")}
        out.update({n: torch.empty_like(v) for n in ("dv", "dw")})
        out["dlog_alpha"] = torch.empty((B, T, H, dk), dtype=torch.float32, device=q.device)
        out["dS0"] = (torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
                      if want_d_initial_state else None)
    if workspace is None:
        if saved:
            raise ValueError("saved=True needs the workspace filled by chunk_fwd(..., train=True)")
        workspace = alloc_workspace(B, T, H, dk, dv, dt, 1, q.device)
    fn = lib().gdr2_chunk_bwd_saved if saved else lib().gdr2_chunk_bwd
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(initial_state),
                              _ptr(d_o), _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                              _ptr(out["dlog_alpha"]), _ptr(out["db"]), _ptr(out["dw"]), _ptr(out.get("dS0")),
                              B, T, H, dk, dv, dt, _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdr2_chunk_bwd_saved" if saved else "gdr2_chunk_bwd", st)
    return out


def workspace_bytes_gva(B, T, H, Hv, dk, dv, dtype_code, for_bwd) -> int:
    return int(lib().gdr2_workspace_bytes_gva(B, T, H, Hv, dk, dv, dtype_code, int(for_bwd)))


def alloc_workspace_gva(B, T, H, Hv, dk, dv, dtype_code, for_bwd, device=None) -> torch.Tensor:
    n = workspace_bytes_gva(B, T, H, Hv, dk, dv, dtype_code, for_bwd)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def chunk_fwd_gva(q, k, v, log_alpha, b, w, initial_state=None, *, output_final_state=True, o=None,
                  final_state=None, workspace=None, stream=None, train=False):
    """gdr2_chunk_fwd_gva (or the _train variant): grouped value heads. q, k, log_alpha, b [B,T,H,dk];
    v, w [B,T,Hv,dv] with Hv a multiple of H; states [B,Hv,dk,dv]. Returns (o [B,T,Hv,dv], final_state)."""
    if stream is not None:
        return _on(stream, chunk_fwd_gva, locals())
    B, T, H, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty((B, T, Hv, dv), dtype=q.dtype, device=q.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
    if not output_final_state:
        final_state = None
    if workspace is None:
        if train:
            raise ValueError("train=True needs the workspace that the backward will read")
        workspace = alloc_workspace_gva(B, T, H, Hv, dk, dv, dt, 0, q.device)
    fn = lib().gdr2_chunk_fwd_train_gva if train else lib().gdr2_chunk_fwd_gva
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(initial_state), _ptr(o),
            _ptr(final_state), B, T, H, Hv, dk, dv, dt, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdr2_chunk_fwd_train_gva" if train else "gdr2_chunk_fwd_gva", st)
    return o, final_state


def chunk_bwd_gva(q, k, v, log_alpha, b, w, initial_state=None, d_o=None, d_final_state=None, *,
                  want_d_initial_state=True, out=None, workspace=None, stream=None, saved=False):
    """gdr2_chunk_bwd_gva (or the _saved variant): returns a dict dq, dk, dlog_alpha, db [B,T,H,dk],
    dv, dw [B,T,Hv,dv], dS0 [B,Hv,dk,dv] (or None)."""
    if stream is not None:
        return _on(stream, chunk_bwd_gva, locals())
    B, T, H, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dt = _dtype_code(q)
    if out is None:
        out = {n: torch.empty_like(q) for n in ("dq", "dk", "db")}
        out.update({n: torch.empty_like(v) for n in ("dv", "dw")})
        out["dlog_alpha"] = torch.empty((B, T, H, dk), dtype=torch.float32, device=q.device)
        out["dS0"] = (torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
                      if want_d_initial_state else None)
    if workspace is None:
        if saved:
            raise ValueError("saved=True needs the workspace filled by chunk_fwd_gva(..., train=True)")
        workspace = alloc_workspace_gva(B, T, H, Hv, dk, dv, dt, 1, q.device)
    fn = lib().gdr2_chunk_bwd_saved_gva if saved else lib().gdr2_chunk_bwd_gva
    st = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(initial_state), _ptr(d_o),
            _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlog_alpha"]),
            _ptr(out["db"]), _ptr(out["dw"]), _ptr(out.get("dS0")), B, T, H, Hv, dk, dv, dt, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gdr2_chunk_bwd_saved_gva" if saved else "gdr2_chunk_bwd_gva", st)
    return out


def workspace_bytes_varlen(N, T, H, dk, dv, dtype_code, for_bwd, Hv=None) -> int:
    """gdr2_workspace_bytes_varlen, or gdr2_workspace_bytes_varlen_gva when Hv (value heads) != H."""
    if Hv is not None and Hv != H:
        return int(lib().gdr2_workspace_bytes_varlen_gva(N, T, H, Hv, dk, dv, dtype_code, int(for_bwd)))
    return int(lib().gdr2_workspace_bytes_varlen(N, T, H, dk, dv, dtype_code, int(for_bwd)))


def alloc_workspace_varlen(N, T, H, dk, dv, dtype_code, for_bwd, device=None, Hv=None) -> torch.Tensor:
    n = workspace_bytes_varlen(N, T, H, dk, dv, dtype_code, for_bwd, Hv)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


def _packed_shape(q, cu_seqlens):
    if q.dim() == 4:
        if q.shape[0] != 1:
            raise ValueError("packed token tensors are [T, H, d] or [1, T, H, d]")
        q = q[0]
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D int32 device tensor of N + 1 offsets")
    T, H, dk = q.shape
    return cu_seqlens.numel() - 1, T, H, dk


def chunk_fwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, initial_state=None, *, output_final_state=True,
                     o=None, final_state=None, workspace=None, stream=None, train=False):
    """gdr2_chunk_fwd_varlen (or the _train variant): packed token tensors [T, H, d] (or [1, T, H, d]),
    cu_seqlens int32 [N + 1] on the device, states [N, Hv, dk, dv]. v and w with more heads than q (Hv =
    G H value heads) select gdr2_chunk_fwd_varlen_gva. Returns (o shaped like v, final_state)."""
    if stream is not None:
        return _on(stream, chunk_fwd_varlen, locals())
    N, T, H, dk = _packed_shape(q, cu_seqlens)
    dv, Hv = v.shape[-1], v.shape[-2]
    dt = _dtype_code(q)
    if o is None:
        o = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    if output_final_state and final_state is None:
        final_state = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=q.device)
    if not output_final_state:
        final_state = None
    if workspace is None:
        if train:
            raise ValueError("train=True needs the workspace that the backward will read")
        workspace = alloc_workspace_varlen(N, T, H, dk, dv, dt, 0, q.device, Hv)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(initial_state), _ptr(o),
            _ptr(final_state), _ptr(cu_seqlens), N, T, H]
    tail = [dk, dv, dt, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)]
    if Hv != H:
        name = "gdr2_chunk_fwd_train_varlen_gva" if train else "gdr2_chunk_fwd_varlen_gva"
        st = getattr(lib(), name)(*args, Hv, *tail)
    else:
        name = "gdr2_chunk_fwd_train_varlen" if train else "gdr2_chunk_fwd_varlen"
        st = getattr(lib(), name)(*args, *tail)
    _check(name, st)
    return o, final_state


def chunk_bwd_varlen(q, k, v, log_alpha, b, w, cu_seqlens, initial_state=None, d_o=None, d_final_state=None, *,
                     want_d_initial_state=True, out=None, workspace=None, stream=None, saved=False):
    """gdr2_chunk_bwd_varlen (or the _saved variant after chunk_fwd_varlen(..., train=True) on the same
    workspace); v and w with more heads than q select the _gva entry points. Returns a dict dq, dk, dv,
    dlog_alpha, db, dw, dS0 ([N, Hv, dk, dv] or None)."""
    if stream is not None:
        return _on(stream, chunk_bwd_varlen, locals())
    N, T, H, dk = _packed_shape(q, cu_seqlens)
    dv, Hv = v.shape[-1], v.shape[-2]
    dt = _dtype_code(q)
    if out is None:
        out = {n: torch.empty_like(q) for n in ("dq", "dk", "db")}
        out.update({n: torch.empty_like(v) for n in ("dv", "dw")})
        out["dlog_alpha"] = torch.empty(log_alpha.shape, dtype=torch.float32, device=q.device)
        out["dS0"] = (torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=q.device)
                      if want_d_initial_state else None)
    if workspace is None:
        if saved:
            raise ValueError("saved=True needs the workspace filled by chunk_fwd_varlen(..., train=True)")
        workspace = alloc_workspace_varlen(N, T, H, dk, dv, dt, 1, q.device, Hv)
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(initial_state), _ptr(d_o),
            _ptr(d_final_state), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlog_alpha"]),
            _ptr(out["db"]), _ptr(out["dw"]), _ptr(out.get("dS0")), _ptr(cu_seqlens), N, T, H]
    tail = [dk, dv, dt, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)]
    if Hv != H:
        name = "gdr2_chunk_bwd_saved_varlen_gva" if saved else "gdr2_chunk_bwd_varlen_gva"
        st = getattr(lib(), name)(*args, Hv, *tail)
    else:
        name = "gdr2_chunk_bwd_saved_varlen" if saved else "gdr2_chunk_bwd_varlen"
        st = getattr(lib(), name)(*args, *tail)
    _check(name, st)
    return out


def gate_prologue_fwd(xq, xk, xf, xb, xw, a, delta, *, neg_eig=False, out=None, stream=None):
    """gdr2_gate_prologue_fwd: q, k (L2-normalised), log_alpha (fp32), b, w from the pre-activations
    [B,T,H,d] and a, delta [H,dk]. Returns a dict q, k, log_alpha, b, w."""
    if stream is not None:
        return _on(stream, gate_prologue_fwd, locals())
    B, T, H, dk = xq.shape
    dv = xw.shape[-1]
    if out is None:
        out = {"q": torch.empty_like(xq), "k": torch.empty_like(xk), "b": torch.empty_like(xb),
               "w": torch.empty_like(xw),
               "log_alpha": torch.empty((B, T, H, dk), dtype=torch.float32, device=xq.device)}
    st = lib().gdr2_gate_prologue_fwd(_ptr(xq), _ptr(xk), _ptr(xf), _ptr(xb), _ptr(xw), _ptr(a), _ptr(delta),
                                      int(neg_eig), _ptr(out["q"]), _ptr(out["k"]), _ptr(out["log_alpha"]),
                                      _ptr(out["b"]), _ptr(out["w"]), B, T, H, dk, dv, _dtype_code(xq),
                                      _stream(stream))
    _check("gdr2_gate_prologue_fwd", st)
    return out


def gate_prologue_bwd(xq, xk, xf, xb, xw, a, delta, dq, dk, dlog_alpha, db, dw, *, neg_eig=False, out=None,
                      workspace=None, stream=None):
    """gdr2_gate_prologue_bwd: returns a dict dxq, dxk, dxf, dxb, dxw, da, ddelta."""
    if stream is not None:
        return _on(stream, gate_prologue_bwd, locals())
    B, T, H, dk_ = xq.shape
    dv = xw.shape[-1]
    dt = _dtype_code(xq)
    if out is None:
        out = {"dxq": torch.empty_like(xq), "dxk": torch.empty_like(xk), "dxf": torch.empty_like(xf),
               "dxb": torch.empty_like(xb), "dxw": torch.empty_like(xw),
               "da": torch.empty((H, dk_), dtype=torch.float32, device=xq.device),
               "ddelta": torch.empty((H, dk_), dtype=torch.float32, device=xq.device)}
    if workspace is None:
        n = int(lib().gdr2_gate_prologue_workspace_bytes(B, T, H, dk_, dv, dt))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=xq.device)
    st = lib().gdr2_gate_prologue_bwd(_ptr(xq), _ptr(xk), _ptr(xf), _ptr(xb), _ptr(xw), _ptr(a), _ptr(delta),
                                      int(neg_eig), _ptr(dq), _ptr(dk), _ptr(dlog_alpha), _ptr(db), _ptr(dw),
                                      _ptr(out["dxq"]), _ptr(out["dxk"]), _ptr(out["dxf"]), _ptr(out["dxb"]),
                                      _ptr(out["dxw"]), _ptr(out["da"]), _ptr(out["ddelta"]), B, T, H, dk_, dv, dt,
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream))
    _check("gdr2_gate_prologue_bwd", st)
    return out


def decode_step(q, k, v, log_alpha, b, w, state, o=None, *, stream=None):
    """gdr2_decode_step: updates `state` in place and returns o [B,H,dv]."""
    if stream is not None:
        return _on(stream, decode_step, locals())
    B, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    st = lib().gdr2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(state), _ptr(o),
                                B, H, dk, dv, _dtype_code(q), _stream(stream))
    _check("gdr2_decode_step", st)
    return o


# ---- the attention half of the hybrid cell: query / key prologue, paged cache, attention of one new token ----

ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_PARTS = range(4)
_ROPE = {"none": ROPE_PLAIN, "linear": ROPE_LINEAR, "base": ROPE_BASE, "parts": ROPE_PARTS}


# A decode step makes several of these calls a layer, and a call's kernels take a few microseconds. So each binding
# below tests its arguments in one expression and names the fault (through the helpers that raise) only when it fails.
_I32, _F32, _F64 = torch.int32, torch.float32, torch.float64


def _shaped(name, t, shape, dtype):
    """`t` contiguous, of this shape (a tuple) and dtype; its device is looked at by _device."""
    if t.shape != shape:
        raise ValueError(f"gdr2: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"gdr2: {name} is {t.dtype}, not {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"gdr2: {name} must be contiguous")
    return t


def _token_rows(name, x, dtype):
    """Token rows [T, H, d] or [B, T, H, d] with contiguous heads and channels and one stride from token to token
    (a view of a fused projection may have a larger one): (tokens, heads, channels, stride in elements)."""
    if x.dtype is not dtype:
        raise TypeError(f"gdr2: {name} is {x.dtype}, not {dtype}")
    shape, strides = x.shape, x.stride()
    if len(shape) == 3:
        T, H, d = shape
        step, hs, ds = strides
    elif len(shape) == 4:
        B, n, H, d = shape
        T = B * n
        bs, step, hs, ds = strides
        if n == 1:
            step = bs
        elif B > 1 and bs != n * step:
            raise ValueError(f"gdr2: the tokens of {name} must have one stride across the batch")
    else:
        raise ValueError(f"gdr2: {name} must be [T, H, d] or [B, T, H, d]")
    if T * H * d == 0:
        raise ValueError(f"gdr2: {name} is empty")
    if (ds != 1 and d > 1) or (hs != d and H > 1):
        raise ValueError(f"gdr2: heads and channels of {name} must be contiguous")
    return T, H, d, step if T > 1 else H * d


def _device(*tensors):
    """The index of the current CUDA device, where every tensor has to be: the library launches there."""
    index = tensors[0].get_device()
    if index < 0:
        raise ValueError("gdr2: tensors must live on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"gdr2: tensors on different devices ({tensors[0].device} and {t.device})")
    if index != torch._C._cuda_getDevice():
        raise ValueError(f"gdr2: tensors on {tensors[0].device}, which is not the current CUDA device")
    return index


_MOST = 2**31 - 1


def _narrow(**sizes):
    """Names the size that the library's 32-bit arguments do not hold."""
    for name, n in sizes.items():
        if not -_MOST <= n <= _MOST:
            raise ValueError(f"gdr2: {name} = {n} is too large")


def _p(t):
    return 0 if t is None else t.data_ptr()


# A call's arguments go over in one record (gdr2_attn_call): ctypes converts 22 arguments one by one in about 2 us, and
# these calls are bound by the host where the work is small (a short attn_decode 13.2 -> 11.8 us, the prologue forward and
# backward 35.6 -> 32.2).
_CALLS = {name: (n, struct.Struct(fields)) for n, (name, fields) in enumerate((
    ("gdr2_attn_prologue_fwd", "4Pif2Pf2i2P5i2qP"),
    ("gdr2_attn_prologue_bwd", "4Pif2Pf2i6P5i4qPNP"),
    ("gdr2_attn_prologue_cache", "5Pif3Pf2i4P9i3qP"),
    ("gdr2_attn_decode", "6Pfi2P9iPNP"),
    ("gdr2_kv_reserve", "7P5iPNP"),
    ("gdr2_kv_fork", "10P7iPNP"),
    ("gdr2_kv_compact", "7P7iPNP")))}


def _call(name, *args):
    n, record = _CALLS[name]
    try:
        packed = record.pack(*args)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"gdr2: an argument of {name} does not fit: {e}") from None
    st = (_lib or lib()).gdr2_attn_call(n, packed, record.size)
    if st != OK:
        raise GDR2Error(name, st)


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


@functools.lru_cache(maxsize=1024)  # one entry for each batch size, table and window in use; a server's come back
def _need(name, args):
    return int(getattr(lib(), name)(*args))


def _scratch(like, workspace, name, *args):
    """(workspace or None, its bytes): the one given, or a fresh one of the size that the query `name` gives for these
    arguments (it depends on them alone); None where the call needs none."""
    if workspace is not None:
        if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
            raise ValueError("gdr2: the workspace must be contiguous and on the tensors' device")
        return workspace, workspace.numel() * workspace.element_size()
    n = _need(name, args)
    if n == 0:
        return None, 0
    return like.new_empty(-(-n // like.element_size())), n


def rope_freqs(rot, base=10000.0, *, scaling="none", factor=1.0, orig_len=0, turns_low=1.0, turns_high=32.0,
               device="cuda"):
    """gdr2_rope_freqs: (freqs, mag), the radians per position of the rot / 2 rotated pairs (float64 tensor on
    `device`) and the magnitude for the prologue's `mag`. scaling: "none", "linear", "base" or "parts"."""
    if scaling not in _ROPE:
        raise ValueError(f"gdr2: unknown scaling {scaling!r}; use one of {sorted(_ROPE)}")
    buf = (_D * max(1, int(rot) // 2))()
    mag = _D(1.0)
    _check("gdr2_rope_freqs", lib().gdr2_rope_freqs(buf, ctypes.byref(mag), int(rot), float(base), _ROPE[scaling],
                                                    float(factor), float(orig_len), float(turns_low),
                                                    float(turns_high)))
    return torch.tensor(list(buf), dtype=torch.float64, device=device), float(mag.value)


def _prologue_checks(xq, xk, gq, gk, pos, freqs, norm):
    dtype = xq.dtype
    dt = _dtype_code(xq)
    T, Hq, d, sq = _token_rows("xq", xq, dtype)
    Tk, Hk, dk, sk = _token_rows("xk", xk, dtype)
    if Tk != T or dk != d:
        raise ValueError("gdr2: xq and xk must have the same tokens and channels")
    if gq is not None and (gq.dtype is not _F32 or gq.shape != (d,) or not gq.is_contiguous()):
        _shaped("gq", gq, (d,), _F32)
    if gk is not None and (gk.dtype is not _F32 or gk.shape != (d,) or not gk.is_contiguous()):
        _shaped("gk", gk, (d,), _F32)
    if not norm and (gq is not None or gk is not None):
        raise ValueError("gdr2: gq and gk are gains of the norm; pass None without it")
    if freqs is None:
        return T, Hq, Hk, d, sq, sk, dt, 0
    if freqs.dtype is not _F64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise TypeError("gdr2: freqs must be a contiguous 1-D float64 tensor")
    if pos is None or pos.dtype is not _I32 or pos.numel() != T or not pos.is_contiguous():
        raise ValueError("gdr2: pos must hold one int32 position for each token")
    return T, Hq, Hk, d, sq, sk, dt, 2 * freqs.numel()


def attn_prologue_fwd(xq, xk, gq=None, gk=None, pos=None, freqs=None, *, norm=True, eps=1e-6, mag=1.0,
                      interleaved=False, out=None, stream=None):
    """gdr2_attn_prologue_fwd: per-head RMS norm (unless norm=False) with gains gq, gk [d] fp32 (None: ones) and
    rotary positions of xq [.., T, Hq, d] and xk [.., T, Hk, d] (views of a fused projection allowed), pos int32 for
    each token and freqs float64 (rope_freqs; None: no rotation). Returns a dict q, k (contiguous)."""
    if stream is not None:
        return _on(stream, attn_prologue_fwd, locals())
    T, Hq, Hk, d, sq, sk, dt, rot = _prologue_checks(xq, xk, gq, gk, pos, freqs, norm)
    if out is None:
        index = _device(xq, xk, gq, gk, pos, freqs)
        q, k = torch.empty_like(xq), torch.empty_like(xk)  # contiguous, whatever the token stride of the inputs
        out = {"q": q, "k": k}
    else:
        q, k = _shaped("q", out["q"], xq.shape, xq.dtype), _shaped("k", out["k"], xk.shape, xq.dtype)
        index = _device(xq, xk, gq, gk, pos, freqs, q, k)
    _call(
        "gdr2_attn_prologue_fwd",
        xq.data_ptr(), xk.data_ptr(), _p(gq), _p(gk), 1 if norm else 0, eps, _p(pos), _p(freqs), mag, rot,
        1 if interleaved else 0, q.data_ptr(), k.data_ptr(), T, Hq, Hk, d, dt, sq, sk, _raw_stream(index))
    return out


def attn_prologue_bwd(xq, xk, gq, gk, pos, freqs, dq, dk, *, norm=True, eps=1e-6, mag=1.0, interleaved=False,
                      out=None, workspace=None, stream=None):
    """gdr2_attn_prologue_bwd: returns a dict dxq, dxk and, with the norm, dgq, dgk [d] fp32 (written for gains of
    None too, as the gradient of a gain of ones). `out` may hold dxq, dxk as views of one fused gradient, and may
    leave dgq, dgk out or None when they are not wanted."""
    if stream is not None:
        return _on(stream, attn_prologue_bwd, locals())
    T, Hq, Hk, d, sq, sk, dt, rot = _prologue_checks(xq, xk, gq, gk, pos, freqs, norm)
    dtype = xq.dtype
    if not (dq.shape == xq.shape and dq.dtype is dtype and dq.is_contiguous() and dk.shape == xk.shape and
            dk.dtype is dtype and dk.is_contiguous()):
        _shaped("dq", dq, xq.shape, dtype), _shaped("dk", dk, xk.shape, dtype)
    index = _device(xq, xk, gq, gk, pos, freqs, dq, dk)
    if out is None:
        dxq, dxk = torch.empty_like(dq), torch.empty_like(dk)
        sdq, sdk = Hq * d, Hk * d
        out = {"dxq": dxq, "dxk": dxk}
        dgq = dgk = None
        if norm:
            dgq = xq.new_empty(d, dtype=_F32)
            dgk = torch.empty_like(dgq)
            out["dgq"], out["dgk"] = dgq, dgk
    else:
        dxq, dxk, dgq, dgk = out["dxq"], out["dxk"], out.get("dgq"), out.get("dgk")
        Tq, hq, eq, sdq = _token_rows("dxq", dxq, dtype)
        Tk, hk, ek, sdk = _token_rows("dxk", dxk, dtype)
        if (Tq, hq, eq) != (T, Hq, d) or (Tk, hk, ek) != (T, Hk, d):
            raise ValueError("gdr2: dxq and dxk must have the shapes of xq and xk")
        for name, g in (("dgq", dgq), ("dgk", dgk)):
            if g is not None:
                _shaped(name, g, (d,), _F32)
        _device(xq, dxq, dxk, dgq, dgk)
    nbytes = 0
    if dgq is not None or dgk is not None:
        workspace, nbytes = _scratch(xq, workspace, "gdr2_attn_prologue_workspace_bytes", d)
    _call(
        "gdr2_attn_prologue_bwd",
        xq.data_ptr(), xk.data_ptr(), _p(gq), _p(gk), 1 if norm else 0, eps, _p(pos), _p(freqs), mag, rot,
        1 if interleaved else 0, dq.data_ptr(), dk.data_ptr(), dxq.data_ptr(), dxk.data_ptr(), _p(dgq), _p(dgk), T, Hq,
        Hk, d, dt, sq, sk, sdq, sdk, _p(workspace), nbytes, _raw_stream(index))
    return out


def _fine(index, dtype, *tensors):
    """Contiguous tensors of one dtype on device `index`."""
    for t in tensors:
        if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != index:
            return False
    return True


def _refuse(dtype, pools, table, **ints):
    """Names what is wrong with a cache's tensors: the pools (of this dtype, None: their own), the table, int32 arrays
    name=(tensor, shape)."""
    if pools is not None:
        k_pages, v_pages = pools
        if k_pages.dim() != 4:
            raise ValueError("gdr2: k_pages must be [num_pages, Hk, page_size, d]")
        _shaped("k_pages", k_pages, k_pages.shape, dtype or k_pages.dtype)
        _shaped("v_pages", v_pages, k_pages.shape, k_pages.dtype)
    if table.dim() != 2:
        raise ValueError("gdr2: table must be [R, P]")
    _shaped("table", table, table.shape, _I32)
    for name, (t, shape) in ints.items():
        if t is not None:
            _shaped(name, t, shape, _I32)
    _device(table, *(pools or ()), *(t for t, _ in ints.values()))


def attn_prologue_cache(xq, xk, xv, gq, gk, seq, pos, freqs, k_pages, v_pages, table, *, norm=True, eps=1e-6,
                        mag=1.0, interleaved=False, q=None, stream=None):
    """gdr2_attn_prologue_cache: the prologue for new tokens xq [T, Hq, d], xk, xv [T, Hk, d]; token t is token
    pos[t] of sequence seq[t] (int32; outside [0, R): padding). Keys and values go to the pools k_pages, v_pages
    [num_pages, Hk, page_size, d] by table int32 [R, P]; q is returned (padding rows as they were; in a fresh q they hold
    no value)."""
    if stream is not None:
        return _on(stream, attn_prologue_cache, locals())
    T, Hq, Hk, d, sq, sk, dt, rot = _prologue_checks(xq, xk, gq, gk, pos, freqs, norm)
    Tv, Hv, dv, sv = _token_rows("xv", xv, xq.dtype)
    if pos is None:
        raise ValueError("gdr2: pos is needed to find a token's page")
    if freqs is None and (pos.dtype is not _I32 or pos.numel() != T or not pos.is_contiguous()):
        raise ValueError("gdr2: pos must hold one int32 position for each token")
    shape, tshape, index = k_pages.shape, table.shape, xq.get_device()
    if not (len(shape) == 4 and v_pages.shape == shape and len(tshape) == 2 and seq.shape == (T,) and
            _fine(index, xq.dtype, k_pages, v_pages) and _fine(index, _I32, table, seq)):
        _refuse(xq.dtype, (k_pages, v_pages), table, seq=(seq, (T,)))
    num, Hp, ps, dp = shape
    R, P = tshape
    if R > _MOST or P > _MOST:
        _narrow(R=R, P=P)
    if Tv != T or Hv != Hk or dv != d or Hp != Hk or dp != d:
        raise ValueError("gdr2: xk, xv and the pools must agree in tokens, heads and channels")
    if q is None:
        _device(xq, xk, xv, gq, gk, pos, freqs)
        q = torch.empty_like(xq)
    else:
        _shaped("q", q, xq.shape, xq.dtype)
        _device(xq, xk, xv, gq, gk, pos, freqs, q)
    _call(
        "gdr2_attn_prologue_cache",
        xq.data_ptr(), xk.data_ptr(), xv.data_ptr(), _p(gq), _p(gk), 1 if norm else 0, eps, seq.data_ptr(),
        pos.data_ptr(), _p(freqs), mag, rot, 1 if interleaved else 0, q.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), table.data_ptr(), T, Hq, Hk, d, R, P, ps, num, dt, sq, sk, sv, _raw_stream(index))
    return q


def attn_decode(q, k_pages, v_pages, table, lens, seq=None, *, scale=None, window=0, want_lse=False, o=None,
                lse=None, workspace=None, stream=None):
    """gdr2_attn_decode: attention of one new token for each row of q [N, Hq, d] over sequence seq[n] (int32 [N];
    None: n) of the cache, its last `window` tokens (0: all), lens int32 [R] with the new token counted. scale: by
    default d^-1/2. Returns o [N, Hq, d], or (o, lse fp32 [N, Hq]) with want_lse or a given lse (slots whose seq is outside
    [0, R) keep their rows; in fresh outputs those hold no value)."""
    if stream is not None:
        return _on(stream, attn_decode, locals())
    dtype, dt = q.dtype, _dtype_code(q)
    qshape, shape, tshape, index = q.shape, k_pages.shape, table.shape, q.get_device()
    if len(qshape) != 3 or not q.is_contiguous():
        raise ValueError("gdr2: q must be a contiguous [N, Hq, d]")
    N, Hq, d = qshape
    if not (len(shape) == 4 and v_pages.shape == shape and len(tshape) == 2 and lens.shape == tshape[:1] and
            (seq is None or (seq.shape == qshape[:1] and _fine(index, _I32, seq))) and
            _fine(index, dtype, k_pages, v_pages) and _fine(index, _I32, table, lens)):
        _refuse(dtype, (k_pages, v_pages), table, lens=(lens, tshape[:1]), seq=(seq, qshape[:1]))
    num, Hk, ps, dp = shape
    R, P = tshape
    if R > _MOST or P > _MOST or not -_MOST <= window <= _MOST:
        _narrow(R=R, P=P, window=window)
    if dp != d:
        raise ValueError("gdr2: q and the pools must agree in channels")
    _device(q, o, lse)
    if o is None:
        o = torch.empty_like(q)
    else:
        _shaped("o", o, qshape, dtype)
    if lse is not None:
        _shaped("lse", lse, (N, Hq), _F32)
    elif want_lse:
        lse = q.new_empty(N, Hq, dtype=_F32)
    workspace, nbytes = _scratch(q, workspace, "gdr2_attn_decode_workspace_bytes", N, Hq, Hk, d, P, ps, window, dt)
    _call(
        "gdr2_attn_decode",
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), _p(seq),
        d ** -0.5 if scale is None else scale, window, o.data_ptr(), _p(lse), N, Hq, Hk, d, R, P, ps, num, dt,
        _p(workspace), nbytes, _raw_stream(index))
    return o if lse is None else (o, lse)


def _given(out, name, like, shape):
    """The bookkeeping output that the caller gave for `name`, or None."""
    t = out.get(name)
    if t is not None:
        _shaped(name, t, shape, _I32)
        if t.get_device() != like.get_device():
            raise ValueError(f"gdr2: {name} is on another device")
    return t


def kv_reserve(table, lens, want, ref, *, page_size, window=0, out=None, workspace=None, stream=None):
    """gdr2_kv_reserve: pages for tokens [lens[r], want[r]) of every sequence (pages behind the window released
    first). Returns (table, ref, missing int32 [1]) after the call; `out` may name them (also the inputs)."""
    if stream is not None:
        return _on(stream, kv_reserve, locals())
    shape, rows, index, num = table.shape, table.shape[:1], table.get_device(), ref.numel()
    if not (len(shape) == 2 and lens.shape == rows and want.shape == rows and ref.dim() == 1 and
            _fine(index, _I32, table, lens, want, ref)):
        _refuse(None, None, table, lens=(lens, rows), want=(want, rows), ref=(ref, (num,)))
    R, P = shape
    if R > _MOST or P > _MOST or num > _MOST or not (-_MOST <= page_size <= _MOST and -_MOST <= window <= _MOST):
        _narrow(R=R, P=P, num_pages=num, page_size=page_size, window=window)
    _device(table)
    t = r = m = None
    if out is not None:
        t, r, m = _given(out, "table", ref, (R, P)), _given(out, "ref", ref, (num,)), _given(out, "missing", ref, (1,))
    t = torch.empty_like(table) if t is None else t
    r = torch.empty_like(ref) if r is None else r
    m = ref.new_empty(1) if m is None else m
    workspace, nbytes = _scratch(ref, workspace, "gdr2_kv_workspace_bytes", R, P, num)
    _call(
        "gdr2_kv_reserve",
        table.data_ptr(), lens.data_ptr(), want.data_ptr(), ref.data_ptr(), t.data_ptr(), r.data_ptr(), m.data_ptr(),
        R, P, page_size, num, window, _p(workspace), nbytes, _raw_stream(index))
    return t, r, m


def kv_fork(table, lens, ref, parent, k_pages, v_pages, *, out=None, workspace=None, stream=None):
    """gdr2_kv_fork: sequence r takes over the content of sequence parent[r] (int32 [R]; r: stays, outside [0, R):
    released). Partly filled last pages are copied in the pools. Returns (table, lens, ref, missing int32 [1])."""
    if stream is not None:
        return _on(stream, kv_fork, locals())
    shape, rows, pool, index, dt = table.shape, table.shape[:1], k_pages.shape, table.get_device(), _dtype_code(k_pages)
    if not (len(shape) == 2 and len(pool) == 4 and v_pages.shape == pool and lens.shape == rows and
            parent.shape == rows and ref.shape == pool[:1] and _fine(index, _I32, table, lens, parent, ref) and
            _fine(index, k_pages.dtype, k_pages, v_pages)):
        _refuse(None, (k_pages, v_pages), table, lens=(lens, rows), parent=(parent, rows), ref=(ref, pool[:1]))
    (R, P), (num, Hk, ps, d) = shape, pool
    if R > _MOST or P > _MOST:
        _narrow(R=R, P=P)
    _device(table)
    t = n = r = m = None
    if out is not None:
        t, n = _given(out, "table", ref, (R, P)), _given(out, "lens", ref, (R,))
        r, m = _given(out, "ref", ref, (num,)), _given(out, "missing", ref, (1,))
    t = torch.empty_like(table) if t is None else t
    n = torch.empty_like(lens) if n is None else n
    r = torch.empty_like(ref) if r is None else r
    m = ref.new_empty(1) if m is None else m
    workspace, nbytes = _scratch(ref, workspace, "gdr2_kv_workspace_bytes", R, P, num)
    _call(
        "gdr2_kv_fork",
        table.data_ptr(), lens.data_ptr(), ref.data_ptr(), parent.data_ptr(), t.data_ptr(), n.data_ptr(), r.data_ptr(),
        m.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), R, P, Hk, ps, d, num, dt, _p(workspace), nbytes,
        _raw_stream(index))
    return t, n, r, m


def kv_compact(table, ref, k_pages, v_pages, *, out=None, workspace=None, stream=None):
    """gdr2_kv_compact: the live pages moved to [0, live). Returns (table, ref, live int32 [1])."""
    if stream is not None:
        return _on(stream, kv_compact, locals())
    shape, pool, index, dt = table.shape, k_pages.shape, table.get_device(), _dtype_code(k_pages)
    if not (len(shape) == 2 and len(pool) == 4 and v_pages.shape == pool and ref.shape == pool[:1] and
            _fine(index, _I32, table, ref) and _fine(index, k_pages.dtype, k_pages, v_pages)):
        _refuse(None, (k_pages, v_pages), table, ref=(ref, pool[:1]))
    (R, P), (num, Hk, ps, d) = shape, pool
    if R > _MOST or P > _MOST:
        _narrow(R=R, P=P)
    _device(table)
    t = r = m = None
    if out is not None:
        t, r, m = _given(out, "table", ref, (R, P)), _given(out, "ref", ref, (num,)), _given(out, "live", ref, (1,))
    t = torch.empty_like(table) if t is None else t
    r = torch.empty_like(ref) if r is None else r
    m = ref.new_empty(1) if m is None else m
    workspace, nbytes = _scratch(ref, workspace, "gdr2_kv_workspace_bytes", R, P, num)
    _call(
        "gdr2_kv_compact",
        table.data_ptr(), ref.data_ptr(), t.data_ptr(), r.data_ptr(), m.data_ptr(), k_pages.data_ptr(),
        v_pages.data_ptr(), R, P, Hk, ps, d, num, dt, _p(workspace), nbytes, _raw_stream(index))
    return t, r, m


def profile_enable(on: bool = True) -> None:
    """Turn per-kernel event timing on or off for later launches (benchmark support)."""
    lib().gdr2_profile_enable(int(bool(on)))


def profile_collect(max_entries: int = 64) -> dict:
    """Wait for recorded launches and return {kernel name: (launches, total ms)}; clears the record."""
    stride = 64
    names = ctypes.create_string_buffer(stride * max_entries)
    launches = (_I * max_entries)()
    ms = (ctypes.c_double * max_entries)()
    dropped = _I(0)
    n = lib().gdr2_profile_collect(names, stride, launches, ms, max_entries, ctypes.byref(dropped))
    if n < 0:
        raise GDR2Error("gdr2_profile_collect", -n)
    out = {}
    for i in range(n):
        nm = names.raw[i * stride:(i + 1) * stride].split(b"\0", 1)[0].decode()
        out[nm] = (int(launches[i]), float(ms[i]))
    if dropped.value:
        out["<dropped>"] = (int(dropped.value), 0.0)
    return out

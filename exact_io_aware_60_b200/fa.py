"""ctypes binding of libfa.so (declared in include/fa.h).

The functions named like the C entry points (``fa_fwd``, ``fa_bwd``, ...) only marshal
arguments: they check shapes and dtypes, take raw device pointers from torch tensors
and pass the current CUDA stream.  Every step of the computation runs in the library's
CUDA kernels.  ``forward`` / ``backward`` additionally allocate the outputs with torch.

The library is loaded on first use.  If ``libfa.so`` is missing, or a call returns an
error, a :class:`FAError` is raised: there is no fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import math
import os
import threading
import warnings
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")


def _load_quick():
    """The compiled binding of the serving calls, or None (the same calls go by ctypes): it is not
    built, or, which is said, it was built for another torch or Python."""
    why = None
    try:
        from . import _fa_binding as quick  # (needs torch's libraries, loaded above)
        if getattr(quick, "built_for", None) == torch.__version__:
            return quick
        why = f"built for torch {getattr(quick, 'built_for', '?')}, this is {torch.__version__}"
    except ImportError as e:
        if os.path.exists(os.path.join(_HERE, "_fa_binding.so")):
            why = str(e)
    if why:
        warnings.warn(f"_fa_binding.so is not used ({why}); the serving calls go by ctypes, some "
                      "5 us of host time each slower.  Build it again: python -m "
                      f"{__package__}.build", RuntimeWarning, stacklevel=2)
    return None


_quick = _load_quick()

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_ERR_SCRATCH_LIMIT = 5
FA_ERR_BAD_PAGE = 6
FA_NOALLOC_SCRATCH_BYTES = 64 << 20
FA_BF16, FA_FP16 = 0, 1

_lock = threading.Lock()
_lib = None
_addr = {}  # of the entry points that _fa_binding calls


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        if _lib is not None:
            detail = _lib.fa_last_cuda_error().decode()
        msg = f"{where}: {fa_strerror(status)} (status {status})"
        if status == FA_ERR_CUDA and detail:
            msg += f": {detail}"
        super().__init__(msg)


def lib():
    """The loaded ctypes library (raises if libfa.so has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise FAError(FA_ERR_UNSUPPORTED,
                              f"libfa.so not found at {LIB_PATH} (build it with "
                              "`python -m exact_io_aware_60_b200.build`)")
            L = ctypes.CDLL(LIB_PATH)
            vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            L.fa_fwd.restype = i
            L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i, vp]
            L.fa_bwd.restype = i
            L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, i,
                                 vp, sz, vp]
            L.fa_bwd_workspace_bytes.restype = sz
            L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
            L.fa_strerror.restype = ctypes.c_char_p
            L.fa_strerror.argtypes = [i]
            L.fa_last_cuda_error.restype = ctypes.c_char_p
            L.fa_last_cuda_error.argtypes = []
            L.fa_get_device_status.restype = i
            L.fa_get_device_status.argtypes = [vp]
            L.fa_version.restype = i
            L.fa_version.argtypes = []
            L.fa_set_timing_events.restype = i
            L.fa_set_timing_events.argtypes = [i, vp, vp]
            L.fa_selftest_wait_timeout.restype = i
            L.fa_selftest_wait_timeout.argtypes = [i, vp]
            L.fa_fwd_blocksparse.restype = i
            L.fa_fwd_blocksparse.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp, i, i,
                                             vp]
            L.fa_bwd_blocksparse.restype = i
            L.fa_bwd_blocksparse.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f,
                                             i, vp, vp, i, i, vp, sz, vp]
            u64, u32 = ctypes.c_ulonglong, ctypes.c_uint
            L.fa_fwd_dropout.restype = i
            L.fa_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, f, u64, u32, i,
                                         vp]
            L.fa_bwd_dropout.restype = i
            L.fa_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp,
                                         f, u64, u32, i, vp, sz, vp]
            L.fa_dropout_mask.restype = i
            L.fa_dropout_mask.argtypes = [i, i, i, f, u64, u32, vp, vp]
            L.fa_fwd_splitkv_workspace_bytes.restype = sz
            L.fa_fwd_splitkv_workspace_bytes.argtypes = [i, i, i, i, i, i]
            L.fa_fwd_splitkv.restype = i
            L.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, i, i, vp, sz,
                                         vp]
            L.fa_fwd_fp8.restype = i
            L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, f, f, f, vp]
            L.fa_bwd_noalloc.restype = i
            L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i,
                                         vp, i, vp]
            L.fa_rope.restype = i
            L.fa_rope.argtypes = [vp] * 4 + [i] * 5 + [vp] * 5 + [i, vp, i, i, f, i, vp]
            L.fa_rope_bwd.restype = i
            L.fa_rope_bwd.argtypes = L.fa_rope.argtypes
            L.fa_kv_append.restype = i
            L.fa_kv_append.argtypes = ([vp] * 6 + [i] * 5 + [vp] * 6 + [i, i, vp, i] + [vp] * 4
                                       + [i, i, f, i, vp])
            L.fa_fwd_paged_workspace_bytes.restype = sz
            L.fa_fwd_paged_workspace_bytes.argtypes = [i] * 5
            L.fa_fwd_paged.restype = i
            L.fa_fwd_paged.argtypes = ([vp] * 5 + [i] * 5 + [vp] * 4 + [i, i, vp, i] + [vp] * 3
                                       + [i, f, i, vp, sz, vp])
            L.fa_schedule_items.restype = i
            L.fa_schedule_items.argtypes = [vp, i, i, vp, vp]
            for n in ("fa_rope", "fa_rope_bwd", "fa_kv_append", "fa_fwd_paged"):
                _addr[n] = ctypes.cast(getattr(L, n), ctypes.c_void_p).value
            _lib = L
    return _lib


def fa_strerror(status: int) -> str:
    if _lib is None:
        return {0: "ok", 1: "invalid argument", 2: "unsupported configuration or device",
                3: "CUDA error", 4: "device-side wait timed out",
                5: "problem needs more scratch than fa_bwd_noalloc's static buffer",
                6: "page number or length outside the paged cache"}.get(
                    status, "unknown status")
    return _lib.fa_strerror(int(status)).decode()


def fa_version() -> int:
    return int(lib().fa_version())


def fa_schedule_items(cost, lists: int):
    """The launchers' static schedule of items with host costs ``cost`` over ``lists``
    lists: (off, ids) as numpy arrays, list c = ids[off[c]:off[c + 1]] (host only)."""
    import numpy as np
    c = np.ascontiguousarray(np.asarray(cost, dtype=np.float32))
    off = np.zeros(int(lists) + 1, dtype=np.uint16)
    ids = np.zeros(max(len(c), 1), dtype=np.uint16)
    rc = lib().fa_schedule_items(c.ctypes.data, len(c), int(lists), off.ctypes.data,
                                 ids.ctypes.data)
    if rc != FA_OK:
        raise FAError(rc, "fa_schedule_items")
    return off, ids[:len(c)]


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise FAError(FA_ERR_INVALID_ARG, f"unsupported dtype {t.dtype}")


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _check(t: torch.Tensor, name: str, shape, dtype):
    if not isinstance(t, torch.Tensor):
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG,
                      f"{name}: expected contiguous {dtype} {tuple(shape)}, got "
                      f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")


def _kv_ptr(kv_len, B):
    if kv_len is None:
        return None
    _check(kv_len, "kv_len", (B,), torch.int32)
    return kv_len.data_ptr()


def fa_fwd(q, k, v, o, lse, *, scale: float, causal: bool = False, kv_len=None,
           stream=None) -> None:
    """Enqueues the forward pass: writes ``o`` ([B,H,N,d]) and ``lse`` ([B,H,N] fp32)."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    rc = lib().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                      B, H, N, d, float(scale), int(bool(causal)), _kv_ptr(kv_len, B),
                      _dtype_code(q), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd")


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, N, d))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, *, scale: float, causal: bool = False,
           kv_len=None, workspace: torch.Tensor, stream=None) -> None:
    """Enqueues the backward pass: writes ``dq``, ``dk``, ``dv``.  ``workspace`` is a
    uint8 CUDA tensor of at least ``fa_bwd_workspace_bytes`` bytes."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG, "workspace must be a contiguous uint8 CUDA tensor")
    rc = lib().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                      lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                      float(scale), int(bool(causal)), _kv_ptr(kv_len, B), _dtype_code(q),
                      workspace.data_ptr(), workspace.numel(), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd")


def _mask_args(block_mask, B, H, N):
    T = (N + 127) // 128
    if not isinstance(block_mask, torch.Tensor) or not block_mask.is_cuda:
        raise FAError(FA_ERR_INVALID_ARG, "block_mask must be a CUDA tensor")
    if block_mask.dtype != torch.uint8 or not block_mask.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG, "block_mask must be a contiguous uint8 tensor")
    if tuple(block_mask.shape) == (T, T):
        return block_mask.data_ptr(), 0
    if tuple(block_mask.shape) == (B, H, T, T):
        return block_mask.data_ptr(), 1
    raise FAError(FA_ERR_INVALID_ARG,
                  f"block_mask shape must be ({T}, {T}) or ({B}, {H}, {T}, {T})")


def fa_fwd_blocksparse(q, k, v, o, lse, block_mask, *, scale: float, causal: bool = False,
                       kv_len=None, stream=None) -> None:
    """Block-sparse forward: ``block_mask`` is a uint8 CUDA tensor [T, T] or [B, H, T, T]
    (T = ceil(N/128)); key tile kt is visible to query tile qt only where it is nonzero."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    mp, per_head = _mask_args(block_mask, B, H, N)
    rc = lib().fa_fwd_blocksparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  lse.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                                  _kv_ptr(kv_len, B), mp, per_head, _dtype_code(q),
                                  _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_blocksparse")


def fa_bwd_blocksparse(q, k, v, o, dout, lse, dq, dk, dv, block_mask, *, scale: float,
                       causal: bool = False, kv_len=None, workspace: torch.Tensor,
                       stream=None) -> None:
    """Block-sparse backward with the same ``block_mask`` as the forward call."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG, "workspace must be a contiguous uint8 CUDA tensor")
    mp, per_head = _mask_args(block_mask, B, H, N)
    rc = lib().fa_bwd_blocksparse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                                  _kv_ptr(kv_len, B), mp, per_head, _dtype_code(q),
                                  workspace.data_ptr(), workspace.numel(),
                                  _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_blocksparse")


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, *, scale: float, causal: bool = False,
                   kv_len=None, stream=None) -> None:
    """Enqueues the backward pass using the library's static scratch instead of a
    caller workspace, for callers that cannot allocate device memory (see include/fa.h:
    problems needing more than FA_NOALLOC_SCRATCH_BYTES of scratch are refused, and
    calls that may overlap on the GPU race on the shared scratch)."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    rc = lib().fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                              dv.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                              _kv_ptr(kv_len, B), _dtype_code(q), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_noalloc")


def fa_fwd_dropout(q, k, v, o, lse, *, scale: float, p_drop: float, seed: int, offset: int = 0,
                   causal: bool = False, kv_len=None, stream=None) -> None:
    """Forward pass with dropout of probability ``p_drop`` on the attention weights; the
    keep mask is drawn from (``seed``, ``offset``) and never stored (see include/fa.h)."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    rc = lib().fa_fwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                              _kv_ptr(kv_len, B), float(p_drop), int(seed), int(offset),
                              _dtype_code(q), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, dout, lse, dq, dk, dv, *, scale: float, p_drop: float, seed: int,
                   offset: int = 0, causal: bool = False, kv_len=None, workspace: torch.Tensor,
                   stream=None) -> None:
    """Backward pass of :func:`fa_fwd_dropout`; give it the same p_drop, seed, offset."""
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        _check(t, name, (B, H, N, d), q.dtype)
    _check(lse, "lse", (B, H, N), torch.float32)
    if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG, "workspace must be a contiguous uint8 CUDA tensor")
    rc = lib().fa_bwd_dropout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                              dv.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                              _kv_ptr(kv_len, B), float(p_drop), int(seed), int(offset),
                              _dtype_code(q), workspace.data_ptr(), workspace.numel(),
                              _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_bwd_dropout")


def fa_dropout_mask(keep, *, p_drop: float, seed: int, offset: int = 0, stream=None) -> None:
    """Writes the keep mask of the dropout calls into ``keep``, a uint8 CUDA tensor
    [B, H, N, N] (1 = kept)."""
    if not isinstance(keep, torch.Tensor) or not keep.is_cuda or keep.dtype != torch.uint8 \
            or not keep.is_contiguous() or keep.dim() != 4 or keep.shape[2] != keep.shape[3]:
        raise FAError(FA_ERR_INVALID_ARG, "keep must be a contiguous uint8 CUDA tensor [B,H,N,N]")
    B, H, N, _ = keep.shape
    rc = lib().fa_dropout_mask(B, H, N, float(p_drop), int(seed), int(offset), keep.data_ptr(),
                               _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_dropout_mask")


def fa_fwd_splitkv_workspace_bytes(B: int, H: int, Nq: int, Nk: int, d: int,
                                   num_splits: int = 0) -> int:
    return int(lib().fa_fwd_splitkv_workspace_bytes(B, H, Nq, Nk, d, num_splits))


def fa_fwd_splitkv(q, k, v, o, lse, *, scale: float, causal: bool = False, kv_len=None,
                   num_splits: int = 0, workspace=None, stream=None) -> None:
    """Inference-shaped forward: q, o [B,H,Nq,d] against k, v [B,H,Nk,d], the key range
    split over CTAs and merged (see include/fa.h).  ``workspace``: uint8 CUDA tensor of
    ``fa_fwd_splitkv_workspace_bytes`` bytes (None allowed when that is 0)."""
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    for name, t, n in (("q", q, Nq), ("k", k, Nk), ("v", v, Nk), ("o", o, Nq)):
        _check(t, name, (B, H, n, d), q.dtype)
    _check(lse, "lse", (B, H, Nq), torch.float32)
    if workspace is not None and (not workspace.is_cuda or workspace.dtype != torch.uint8
                                  or not workspace.is_contiguous()):
        raise FAError(FA_ERR_INVALID_ARG, "workspace must be a contiguous uint8 CUDA tensor")
    rc = lib().fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              lse.data_ptr(), B, H, Nq, Nk, d, float(scale), int(bool(causal)),
                              _kv_ptr(kv_len, B), int(num_splits), _dtype_code(q),
                              None if workspace is None else workspace.data_ptr(),
                              0 if workspace is None else workspace.numel(),
                              _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_splitkv")


def forward_splitkv(q, k, v, *, scale: Optional[float] = None, causal: bool = False,
                    kv_len=None, num_splits: int = 0, stream=None):
    """Allocates ``o``, ``lse`` and the workspace with torch and runs :func:`fa_fwd_splitkv`."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    B, H, Nq, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    n = fa_fwd_splitkv_workspace_bytes(B, H, Nq, k.shape[2], d, num_splits)
    ws = torch.empty(n, dtype=torch.uint8, device=q.device) if n > 0 else None
    fa_fwd_splitkv(q, k, v, o, lse, scale=scale, causal=causal, kv_len=kv_len,
                   num_splits=num_splits, workspace=ws, stream=stream)
    return o, lse


def fa_fwd_fp8(q8, k8, v8, o, lse, *, scale: float, q_scale: float, k_scale: float,
               v_scale: float, causal: bool = False, kv_len=None, stream=None) -> None:
    """FP8 forward: q8, k8, v8 are E4M3 tensors (torch.float8_e4m3fn, or their uint8 bytes)
    [B,H,N,128] with per-tensor scale factors; writes bf16 ``o`` and fp32 ``lse``."""
    B, H, N, d = q8.shape
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        if not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (B, H, N, d) \
                or t.element_size() != 1:
            raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a contiguous 1-byte CUDA tensor "
                                              f"of shape {(B, H, N, d)}")
    _check(o, "o", (B, H, N, d), torch.bfloat16)
    _check(lse, "lse", (B, H, N), torch.float32)
    rc = lib().fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(), o.data_ptr(),
                          lse.data_ptr(), B, H, N, d, float(scale), int(bool(causal)),
                          _kv_ptr(kv_len, B), float(q_scale), float(k_scale), float(v_scale),
                          _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_fp8")


# ------------------------------------------------------------------ rotary positions

@dataclasses.dataclass(frozen=True)
class RopePlan:
    """What :func:`fa_rope` and :func:`fa_kv_append` rotate by (made by :func:`rope_plan`).

    ``turns``: int64 CUDA tensor [rot_dim / 2], each pair's angle per position as a fraction
    of a turn in units of 2^-64 (the bits of the unsigned value of include/fa.h)."""
    turns: torch.Tensor
    rot_dim: int
    interleaved: bool
    magnitude: float


def rope_frequencies(rot_dim: int, *, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, original_length: Optional[int] = None,
                     beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(f, magnitude): the angle per position of each pair, a list of rot_dim / 2 floats in
    64 bits, and the factor of the rotated elements.

    f_i = base^(-2 i / rot_dim), scaled for contexts ``factor`` times as long by

    * ``"linear"`` (position interpolation): f_i / factor;
    * ``"ntk"``: base multiplied by factor^(rot_dim / (rot_dim - 2)), so that the slowest
      pair is scaled by 1 / factor and the fastest not at all;
    * ``"yarn"`` (YaRN, Peng et al. 2023): pairs that turn more than ``beta_fast`` times
      within ``original_length`` keep f_i, those below ``beta_slow`` get f_i / factor, a
      linear ramp in between; the magnitude is 0.1 ln(factor) + 1."""
    if rot_dim < 2 or rot_dim % 2 or not (math.isfinite(base) and base > 0.0):
        raise FAError(FA_ERR_INVALID_ARG, "rope_frequencies: rot_dim even and >= 2, base > 0")
    if not (math.isfinite(factor) and factor >= 1.0):
        raise FAError(FA_ERR_INVALID_ARG, "rope_frequencies: factor must be finite and >= 1")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise FAError(FA_ERR_INVALID_ARG, f"rope_frequencies: unknown scaling {scaling!r}")
    if scaling == "ntk":
        if rot_dim == 2:
            raise FAError(FA_ERR_INVALID_ARG, "rope_frequencies: ntk needs rot_dim > 2")
        try:
            base = base * factor ** (rot_dim / (rot_dim - 2))
        except OverflowError:
            base = math.inf
        if math.isinf(base):
            raise FAError(FA_ERR_INVALID_ARG, "rope_frequencies: ntk's base overflows")
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        if original_length is None or original_length < 1 or not beta_fast > beta_slow:
            raise FAError(FA_ERR_INVALID_ARG, "rope_frequencies: yarn needs original_length >= 1 "
                                              "and beta_fast > beta_slow")
        out = []
        for x in f:
            r = original_length * x / (2.0 * math.pi)
            keep = min(max((r - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0)
            out.append((1.0 - keep) * x / factor + keep * x)
        return out, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope_plan(rot_dim: int, *, layout: str = "half", base: float = 10000.0, scaling: str = "none",
              factor: float = 1.0, original_length: Optional[int] = None,
              beta_fast: float = 32.0, beta_slow: float = 1.0, frequencies=None,
              magnitude: Optional[float] = None, device=None) -> RopePlan:
    """A rotation plan, made once and kept.  ``layout``: "half" (pairs (i, i + rot_dim / 2))
    or "interleaved" (pairs (2 i, 2 i + 1)).  The frequencies are :func:`rope_frequencies`'s,
    or ``frequencies``: rot_dim / 2 angles per position in radians; ``magnitude`` overrides
    the scaling's factor of the rotated elements."""
    if layout not in ("half", "interleaved"):
        raise FAError(FA_ERR_INVALID_ARG, f"rope_plan: unknown layout {layout!r}")
    if rot_dim < 16 or rot_dim % 16:
        raise FAError(FA_ERR_UNSUPPORTED, "rope_plan: rot_dim must be a positive multiple of 16")
    if frequencies is None:
        freq, mag = rope_frequencies(rot_dim, base=base, scaling=scaling, factor=factor,
                                     original_length=original_length, beta_fast=beta_fast,
                                     beta_slow=beta_slow)
    else:
        freq, mag = [float(x) for x in frequencies], 1.0
        if len(freq) != rot_dim // 2 or not all(math.isfinite(x) for x in freq):
            raise FAError(FA_ERR_INVALID_ARG, "rope_plan: frequencies must be rot_dim / 2 finite "
                                              "numbers")
    mag = mag if magnitude is None else float(magnitude)
    if not (math.isfinite(mag) and mag > 0.0):
        raise FAError(FA_ERR_INVALID_ARG, "rope_plan: magnitude must be finite and > 0")
    turns = []
    for x in freq:
        # (whole turns drop out first, exactly: any finite angle has its 64 bits)
        u = int(round(math.fmod(x / (2.0 * math.pi), 1.0) * 2.0 ** 64)) % (1 << 64)
        turns.append(u - (1 << 64) if u >= 1 << 63 else u)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return RopePlan(torch.tensor(turns, dtype=torch.int64, device=device), rot_dim,
                    layout == "interleaved", mag)


_I3 = ctypes.c_longlong * 3
_CODES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # (no Stream object made)


def _stream_of(index: int, stream) -> int:
    """The caller's stream, or device ``index``'s current one."""
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_stream is not None:
        return _raw_stream(index)
    return int(torch.cuda.current_stream(index).cuda_stream)


def _on_device(index: int, fn, args):
    """``fn(*args)`` with the tensors' device current (it makes no difference to the caller's)."""
    before = torch.cuda.current_device()
    if before == index:
        return fn(*args)
    torch.cuda.set_device(index)
    try:
        return fn(*args)
    finally:
        torch.cuda.set_device(before)


def _main(t, name: str):
    """(shape, dtype, device index, dtype code) of a call's first tensor, [.., .., .., d]."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4:
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a 4-dimensional CUDA tensor")
    code = _CODES.get(t.dtype)
    if code is None:
        raise FAError(FA_ERR_INVALID_ARG, f"unsupported dtype {t.dtype}")
    return t.shape, t.dtype, t.get_device(), code


def _rows(t, name: str, shape, dtype, index: int):
    """Checks a [.., .., .., d] tensor with d contiguous; its strides for the library (None if
    contiguous)."""
    if not isinstance(t, torch.Tensor):
        raise FAError(FA_ERR_INVALID_ARG, f"{name} must be a torch.Tensor")
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise FAError(FA_ERR_INVALID_ARG,
                      f"{name}: expected {dtype} {tuple(shape)} on cuda:{index}, got {t.dtype} "
                      f"{tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return None
    st = t.stride()
    if st[3] != 1:
        raise FAError(FA_ERR_INVALID_ARG, f"{name}: the last dimension must be contiguous")
    return _I3(st[0], st[1], st[2])


def _ints(t, name: str, shapes, index: int, dtype=torch.int32):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index \
            or t.shape not in shapes or not t.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG,
                      f"{name} must be a contiguous {dtype} tensor on cuda:{index}, shape "
                      + " or ".join(str(s) for s in shapes))
    return t.data_ptr()


def _plan_args(plan, index: int):
    if not isinstance(plan, RopePlan):
        raise FAError(FA_ERR_INVALID_ARG, "the rotation must be a RopePlan (see rope_plan)")
    turns = _ints(plan.turns, "plan.turns", ((plan.rot_dim // 2,),), index, torch.int64)
    return turns, plan.rot_dim, int(plan.interleaved), plan.magnitude


def _quick_call(fn, where, *args) -> bool:
    """A call through _fa_binding; False where it is not plain (see csrc/binding.cpp)."""
    rc = fn(_addr.get(where) or (lib() and _addr[where]), *args)
    if rc is None:
        return False
    if rc != FA_OK:
        raise FAError(rc, where)
    return True


def _handle(stream):
    return None if stream is None else int(stream.cuda_stream)


def _rope_call(where, x, x_out, plan, y, y_out, positions, stream, names):
    if _quick is not None and isinstance(plan, RopePlan) and _quick_call(
            _quick.rope, where, x, x_out, y, y_out, positions, plan.turns, plan.rot_dim,
            plan.interleaved, plan.magnitude, _handle(stream)):
        return
    fn = getattr(lib(), where)
    shape, dtype, index, code = _main(x, names[0])
    B, H, N, d = shape
    xs = None if x.is_contiguous() else _rows(x, names[0], shape, dtype, index)
    xos = _rows(x_out, names[1], shape, dtype, index)
    yp = yop = ys = yos = None
    Hk = 0
    if y is not None:
        if not isinstance(y, torch.Tensor) or y.dim() != 4 or y_out is None:
            raise FAError(FA_ERR_INVALID_ARG, f"{names[2]} and {names[3]} go together, both "
                                              "4-dimensional tensors")
        ysh = y.shape
        Hk = ysh[1]
        if ysh != (B, Hk, N, d):
            raise FAError(FA_ERR_INVALID_ARG, f"{names[2]}: expected {(B, 'Hk', N, d)}, got "
                                              f"{tuple(ysh)}")
        ys = _rows(y, names[2], ysh, dtype, index)
        yos = _rows(y_out, names[3], ysh, dtype, index)
        yp, yop = y.data_ptr(), y_out.data_ptr()
    elif y_out is not None:
        raise FAError(FA_ERR_INVALID_ARG, f"{names[2]} and {names[3]} go together")
    pp, per_batch = None, 0
    if positions is not None:
        pp = _ints(positions, "positions", ((N,), (B, N)), index)
        per_batch = positions.dim() - 1
    turns, rot, inter, mag = _plan_args(plan, index)
    rc = _on_device(index, fn, (x.data_ptr(), x_out.data_ptr(), yp, yop, B, H, Hk, N, d, xs, xos,
                                ys, yos, pp, per_batch, turns, rot, inter, mag, code,
                                _stream_of(index, stream)))
    if rc != FA_OK:
        raise FAError(rc, where)


def fa_rope(q, q_out, plan: RopePlan, *, k=None, k_out=None, positions=None, stream=None) -> None:
    """Rotary positions: writes ``q_out`` [B,H,N,d] (and ``k_out`` [B,Hk,N,d]) from ``q`` (and
    ``k``) in one launch; ``q_out`` may be ``q``.  Strided views with a contiguous last
    dimension are taken as they are.  ``positions``: int32 [N] or [B,N], None for 0 .. N-1."""
    _rope_call("fa_rope", q, q_out, plan, k, k_out, positions, stream,
               ("q", "q_out", "k", "k_out"))


def fa_rope_bwd(dq_rot, dq, plan: RopePlan, *, k=None, k_out=None, positions=None,
                stream=None) -> None:
    """Backward pass of :func:`fa_rope`: gradients of its inputs from those of its outputs.
    ``dq_rot`` -> ``dq``, and ``k`` (the gradient of the rotated keys) -> ``k_out``."""
    _rope_call("fa_rope_bwd", dq_rot, dq, plan, k, k_out, positions, stream,
               ("dq_rot", "dq", "k", "k_out"))


# ------------------------------------------------------------------ paged cache

def _cache_args(k_cache, v_cache, block_table, cache_len, new_len, B, Hk, d, dtype, index):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise FAError(FA_ERR_INVALID_ARG, "k_cache must be a [pages, Hk, page_size, d] tensor")
    shape = k_cache.shape
    P, hk, page, dc = shape
    if (Hk and hk != Hk) or dc != d:
        raise FAError(FA_ERR_INVALID_ARG, f"k_cache: expected [pages, {Hk or 'Hk'}, page_size, {d}], "
                                          f"got {tuple(shape)}")
    ks = _rows(k_cache, "k_cache", shape, dtype, index)
    vs = _rows(v_cache, "v_cache", shape, dtype, index)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise FAError(FA_ERR_INVALID_ARG, "block_table must be an int32 [B, max_blocks] tensor")
    blocks = block_table.shape[1]
    table = _ints(block_table, "block_table", ((B, blocks),), index)
    held = _ints(cache_len, "cache_len", ((B,),), index)
    new = None if new_len is None else _ints(new_len, "new_len", ((B,),), index)
    return ks, vs, P, hk, page, table, blocks, held, new


def fa_kv_append(k, v, k_cache, v_cache, block_table, cache_len, *, new_len=None,
                 rope: Optional[RopePlan] = None, positions=None, q=None, q_out=None,
                 stream=None) -> None:
    """Appends new keys and values ``k``, ``v`` [B,Hk,T,d] to a paged cache [pages,Hk,page_size,d],
    keys (and queries ``q`` -> ``q_out`` [B,H,T,d]) rotated by ``rope`` on the way.  Token t
    of sequence b goes to slot ``cache_len[b] + t`` (see include/fa.h); the lengths are not
    advanced.  ``new_len``: int32 [B], None for T each; ``positions``: int32 [B,T], None for
    the slots' own.  Strided views with a contiguous last dimension are taken as they are."""
    if _quick is not None and (rope is None or isinstance(rope, RopePlan)) and _quick_call(
            _quick.append, "fa_kv_append", k, v, k_cache, v_cache, block_table, cache_len, new_len,
            q, q_out, positions, *((None, 0, False, 1.0) if rope is None else
                                   (rope.turns, rope.rot_dim, rope.interleaved, rope.magnitude)),
            _handle(stream)):
        return
    shape, dtype, index, code = _main(k, "k")
    B, Hk, T, d = shape
    ks = None if k.is_contiguous() else _rows(k, "k", shape, dtype, index)
    vs = _rows(v, "v", shape, dtype, index)
    kcs, vcs, P, _, page, table, blocks, held, new = _cache_args(
        k_cache, v_cache, block_table, cache_len, new_len, B, Hk, d, dtype, index)
    qp = qop = qs = qos = None
    H = 0
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 4 or q_out is None:
            raise FAError(FA_ERR_INVALID_ARG, "q and q_out go together, both 4-dimensional tensors")
        qsh = q.shape
        H = qsh[1]
        if qsh != (B, H, T, d):
            raise FAError(FA_ERR_INVALID_ARG, f"q: expected {(B, 'H', T, d)}, got {tuple(qsh)}")
        qs = _rows(q, "q", qsh, dtype, index)
        qos = _rows(q_out, "q_out", qsh, dtype, index)
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise FAError(FA_ERR_INVALID_ARG, "q and q_out go together")
    pp = None if positions is None else _ints(positions, "positions", ((B, T),), index)
    turns, rot, inter, mag = (None, 0, 0, 1.0) if rope is None else _plan_args(rope, index)
    rc = _on_device(index, lib().fa_kv_append, (
        k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), qp, qop, B, H, Hk, T, d,
        ks, vs, qs, qos, kcs, vcs, P, page, table, blocks, held, new, pp, turns, rot, inter, mag,
        code, _stream_of(index, stream)))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv_append")


def fa_fwd_paged_workspace_bytes(B: int, H: int, Hk: int, T: int, d: int) -> int:
    return int(lib().fa_fwd_paged_workspace_bytes(B, H, Hk, T, d))


def fa_fwd_paged(q, k_cache, v_cache, block_table, cache_len, o, lse, *, scale: float,
                 new_len=None, tree_mask=None, workspace: torch.Tensor, stream=None) -> None:
    """Attention of the new tokens ``q`` [B,H,T,d] over a paged cache that already holds their
    keys and values: writes ``o`` [B,H,T,d] and ``lse`` [B,H,T].  ``tree_mask``: uint8 [T,T] or
    [B,T,T] (row = token, column = new key it sees), None for a chain.  ``workspace``: uint8
    CUDA tensor of ``fa_fwd_paged_workspace_bytes`` bytes.  See include/fa.h."""
    if _quick is not None and _quick_call(
            _quick.paged, "fa_fwd_paged", q, k_cache, v_cache, block_table, cache_len, new_len, o,
            lse, tree_mask, workspace, scale, _handle(stream)):
        return
    shape, dtype, index, code = _main(q, "q")
    B, H, T, d = shape
    qs = None if q.is_contiguous() else _rows(q, "q", shape, dtype, index)
    os_ = _rows(o, "o", shape, dtype, index)
    kcs, vcs, P, Hk, page, table, blocks, held, new = _cache_args(
        k_cache, v_cache, block_table, cache_len, new_len, B, 0, d, dtype, index)
    lp = _ints(lse, "lse", ((B, H, T),), index, torch.float32)
    tp, per_batch = None, 0
    if tree_mask is not None:
        tp = _ints(tree_mask, "tree_mask", ((T, T), (B, T, T)), index, torch.uint8)
        per_batch = tree_mask.dim() - 2
    if not isinstance(workspace, torch.Tensor) or workspace.dtype is not torch.uint8 \
            or workspace.get_device() != index or not workspace.is_contiguous():
        raise FAError(FA_ERR_INVALID_ARG,
                      f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    rc = _on_device(index, lib().fa_fwd_paged, (
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), o.data_ptr(), lp, B, H, Hk, T, d, qs,
        os_, kcs, vcs, P, page, table, blocks, held, new, tp, per_batch, float(scale), code,
        workspace.data_ptr(), workspace.numel(), _stream_of(index, stream)))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_paged")


def fa_set_timing_events(which: int, start=None, stop=None) -> None:
    """Profiling hook: record torch.cuda.Event ``start``/``stop`` around every launch of
    the forward kernel (which=0) or the backward main kernel (which=1); None switches it
    off.  The events must have been recorded once (so that they exist)."""
    h0 = None if start is None else start.cuda_event
    h1 = None if stop is None else stop.cuda_event
    rc = lib().fa_set_timing_events(int(which), h0, h1)
    if rc != FA_OK:
        raise FAError(rc, "fa_set_timing_events")


def fa_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Enqueues the bounded-wait self-test kernel (see include/fa.h)."""
    rc = lib().fa_selftest_wait_timeout(int(limit_us), _stream_handle(stream))
    if rc != FA_OK:
        raise FAError(rc, "fa_selftest_wait_timeout")


def fa_get_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status word."""
    return int(lib().fa_get_device_status(_stream_handle(stream)))


# ------------------------------------------------------------------ conveniences

def forward(q, k, v, *, scale: Optional[float] = None, causal: bool = False, kv_len=None,
            stream=None):
    """Allocates ``o`` and ``lse`` with torch and runs :func:`fa_fwd`."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, scale=scale, causal=causal, kv_len=kv_len, stream=stream)
    return o, lse


def workspace_for(q) -> torch.Tensor:
    B, H, N, d = q.shape
    return torch.empty(fa_bwd_workspace_bytes(B, H, N, d), dtype=torch.uint8, device=q.device)


def backward(q, k, v, o, dout, lse, *, scale: Optional[float] = None, causal: bool = False,
             kv_len=None, workspace=None, stream=None):
    """Allocates ``dq``, ``dk``, ``dv`` (and the workspace if not given) and runs
    :func:`fa_bwd`."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = workspace_for(q)
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, scale=scale, causal=causal, kv_len=kv_len,
           workspace=workspace, stream=stream)
    return dq, dk, dv


@contextlib.contextmanager
def _allocating(t, name: str, stream):
    """The helpers below allocate on the tensors' device and in the call's stream, so that a
    temporary's memory is reused only after the kernels that still read it."""
    _main(t, name)
    with torch.cuda.device(t.get_device()):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def rope(q, plan: RopePlan, *, k=None, positions=None, stream=None):
    """Allocates the outputs with torch and runs :func:`fa_rope`; returns ``q_rot``, or
    ``(q_rot, k_rot)`` with keys."""
    with _allocating(q, "q", stream):
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        k_out = None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format)
        fa_rope(q, q_out, plan, k=k, k_out=k_out, positions=positions, stream=stream)
    return q_out if k is None else (q_out, k_out)


def rope_backward(dq_rot, plan: RopePlan, *, dk_rot=None, positions=None, stream=None):
    """Allocates the outputs with torch and runs :func:`fa_rope_bwd`; returns ``dq``, or
    ``(dq, dk)``."""
    with _allocating(dq_rot, "dq_rot", stream):
        dq = torch.empty_like(dq_rot, memory_format=torch.contiguous_format)
        dk = None if dk_rot is None else torch.empty_like(dk_rot,
                                                          memory_format=torch.contiguous_format)
        fa_rope_bwd(dq_rot, dq, plan, k=dk_rot, k_out=dk, positions=positions, stream=stream)
    return dq if dk_rot is None else (dq, dk)


def forward_rope(q, k, v, plan: RopePlan, *, positions=None, scale: Optional[float] = None,
                 causal: bool = False, kv_len=None, stream=None):
    """:func:`fa_rope` of q and k, then :func:`forward`: returns ``(o, lse, q_rot, k_rot)``,
    the last two for :func:`backward_rope`."""
    with _allocating(q, "q", stream):
        q_rot, k_rot = rope(q, plan, k=k, positions=positions, stream=stream)
        o, lse = forward(q_rot, k_rot, v, scale=scale, causal=causal, kv_len=kv_len, stream=stream)
    return o, lse, q_rot, k_rot


def backward_rope(q_rot, k_rot, v, o, dout, lse, plan: RopePlan, *, positions=None,
                  scale: Optional[float] = None, causal: bool = False, kv_len=None,
                  workspace=None, stream=None):
    """Gradients of :func:`forward_rope`'s q, k, v: :func:`backward`, then dq and dk turned back
    in place."""
    with _allocating(q_rot, "q_rot", stream):
        dq, dk, dv = backward(q_rot, k_rot, v, o, dout, lse, scale=scale, causal=causal,
                              kv_len=kv_len, workspace=workspace, stream=stream)
        fa_rope_bwd(dq, dq, plan, k=dk, k_out=dk, positions=positions, stream=stream)
    return dq, dk, dv


def paged_workspace_for(q, Hk: int, stream=None) -> torch.Tensor:
    """A workspace for :func:`fa_fwd_paged` calls of q's shape with ``Hk`` key/value heads."""
    B, H, T, d = q.shape
    with _allocating(q, "q", stream):
        return torch.empty(fa_fwd_paged_workspace_bytes(B, H, Hk, T, d), dtype=torch.uint8,
                           device=q.device)


def forward_paged(q, k_cache, v_cache, block_table, cache_len, *, scale: Optional[float] = None,
                  new_len=None, tree_mask=None, workspace=None, stream=None):
    """Allocates ``o``, ``lse`` (and the workspace if not given) with torch and runs
    :func:`fa_fwd_paged`."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    with _allocating(q, "q", stream):
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = paged_workspace_for(q, k_cache.shape[1], stream)
        fa_fwd_paged(q, k_cache, v_cache, block_table, cache_len, o, lse, scale=scale,
                     new_len=new_len, tree_mask=tree_mask, workspace=workspace, stream=stream)
    return o, lse


def step_paged(q, k, v, k_cache, v_cache, block_table, cache_len, *,
               rope: Optional[RopePlan] = None, positions=None, scale: Optional[float] = None,
               new_len=None, tree_mask=None, workspace=None, stream=None):
    """A serving step's attention: :func:`fa_kv_append` of the new tokens (q and k rotated by
    ``rope``), then :func:`forward_paged` over the cache.  Returns ``(o, lse)``; the caller
    advances ``cache_len`` once the tokens are accepted."""
    with _allocating(q, "q", stream):
        q_rot = None
        if rope is not None:
            q_rot = torch.empty_like(q, memory_format=torch.contiguous_format)
        fa_kv_append(k, v, k_cache, v_cache, block_table, cache_len, new_len=new_len, rope=rope,
                     positions=positions, q=None if rope is None else q, q_out=q_rot,
                     stream=stream)
        return forward_paged(q if rope is None else q_rot, k_cache, v_cache, block_table,
                             cache_len, scale=scale, new_len=new_len, tree_mask=tree_mask,
                             workspace=workspace, stream=stream)

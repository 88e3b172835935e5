"""Thin ctypes binding of ``libtaylor_attn.so`` (include/taylor_attn.h).

Argument marshalling only: shapes, dtypes, device and contiguity are checked,
raw pointers and the current CUDA stream are passed through, and a non-zero
status becomes :class:`TaylorAttnError`.  Every step of the computation runs
in the library's CUDA kernels; there is no fallback.  The functions carry the
C names; shape arguments (B, H, N, d_k, d_v) are read from the tensors.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional, Tuple

import numpy as np
import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtaylor_attn.so")

TAYLOR_OK = 0
TAYLOR_ERR_INVALID_ARG = -1
TAYLOR_ERR_UNSUPPORTED = -2
TAYLOR_ERR_MISALIGNED = -3
TAYLOR_ERR_CUDA = -4
TAYLOR_ERR_OUT_OF_MEMORY = -5
TAYLOR_ERR_SCRATCH_LIMIT = -6
TAYLOR_ERR_TIMEOUT = -7

# name -> (restype, argtypes); the exported surface of the header
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_I64 = ctypes.c_int64
_QK = [_P, _P, _P, _I64, _P, _I, _I]    # q_weight, k_weight, positions, pos0, freqs, rot, interleaved
_SIZES = [_I] * 5                       # B, N, Hq, Hk, d
SIGNATURES = {
    "taylor_attn_strerror": (ctypes.c_char_p, [_I]),
    "taylor_attn_version": (_I, []),
    "taylor_attn_num_features": (_I64, [_I, _I]),
    "taylor_attn_state_stride": (_I64, [_I, _I, _I]),
    "taylor_attn_feature_index": (_I, [_I, _I, _P, _P]),
    "taylor_attn_feature_map": (_I, [_P, _P, _I64, _I, _I, _F, _I, _P]),
    "taylor_attn_prefill": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_prefill_f32": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_prefill_from_state": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_prefill_from_state_f32": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_decode": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_decode_f32": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_centred_decode": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_centred_decode_f32": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_centred_prefill": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_centred_prefill_f32": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_state_merge": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "taylor_attn_qk_norm_rope": (_I, [_P, _P, *_QK, _P, _P, *_SIZES, _P, _P, _F, _P]),
    "taylor_attn_qk_norm_rope_f32": (_I, [_P, _P, *_QK, _P, _P, *_SIZES, _P, _P, _F, _P]),
    "taylor_attn_qk_norm_rope_backward":
        (_I, [_P, _P, _P, _P, *_QK, _P, _P, _P, _P, *_SIZES, _P, _P, _P, _P, _F, _P]),
    "taylor_attn_qk_norm_rope_backward_f32":
        (_I, [_P, _P, _P, _P, *_QK, _P, _P, _P, _P, *_SIZES, _P, _P, _P, _P, _F, _P]),
    "taylor_attn_gated_scan": (_I, [*[_P] * 6, *[_I] * 3, _P, _P, _I, _P]),
    "taylor_attn_gated_scan_f32": (_I, [*[_P] * 6, *[_I] * 3, _P, _P, _I, _P]),
    "taylor_attn_gated_scan_backward": (_I, [*[_P] * 10, *[_I] * 3, *[_P] * 4, _I, _P]),
    "taylor_attn_gated_scan_backward_f32": (_I, [*[_P] * 10, *[_I] * 3, *[_P] * 4, _I, _P]),
    "taylor_attn_gated_step": (_I, [*[_P] * 5, _I, _I, _I64, _I64, _I, _P]),
    "taylor_attn_gated_step_f32": (_I, [*[_P] * 5, _I, _I, _I64, _I64, _I, _P]),
    "taylor_attn_shared_prefix_decode": (_I, [*[_P] * 8, *[_I] * 6, _F, _P]),
    "taylor_attn_shared_prefix_decode_f32": (_I, [*[_P] * 8, *[_I] * 6, _F, _P]),
    "taylor_attn_prefill_f32_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "taylor_attn_prefill_noalloc_scratch_floats": (_I64, []),
    "taylor_attn_device_errors": (_I, [_I, _P]),
    "taylor_attn_release_workspace": (_I, []),
    "taylor_attn_selftest_bounded_wait": (_I, [ctypes.c_uint, _P]),
    "taylor_attn_timing_enable": (_I, [_I]),
    "taylor_attn_timing_read": (_I, [_I, _P, _P, _P]),
}

_lib = None


class TaylorAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status}: {strerror(status)}")


def lib() -> ctypes.CDLL:
    """Load the library once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m recurrent_states_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().taylor_attn_strerror(int(status)).decode()


def _check(rc: int, where: str) -> None:
    if rc != TAYLOR_OK:
        raise TaylorAttnError(rc, where)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, device=None, shape=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _on(t: torch.Tensor, stream):
    """Context in which t's device is the current one and `stream` (None: that
    device's current stream) its current stream, so that what is allocated in
    it belongs to the stream the kernels run on."""
    if stream is None:
        return torch.cuda.device(t.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream)
                  else torch.cuda.default_stream(t.device))
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def _elsewhere(t: torch.Tensor, stream) -> bool:
    """Whether a call on t has to be made in the context _on(t, stream): another
    device than the current one, or a stream that was given."""
    if not t.is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    return stream is not None or t.get_device() != torch.cuda.current_device()


# The current stream's handle of a device; the public call makes a Stream
# object first, which takes longer than a small kernel's launch.
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _fits(name: str, *sizes: int) -> None:
    """Refuses sizes that are no C int: ctypes would cut them to their low 32 bits."""
    if max(sizes) > 0x7fffffff:
        raise TaylorAttnError(TAYLOR_ERR_UNSUPPORTED, name)


def _want(t: torch.Tensor, name: str, dtype, dev: int, shape) -> None:
    """_need against a device's index; the checks in their quickest form."""
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        _need(t, name, dtype, torch.device("cuda", dev), shape)


def _rows(t: torch.Tensor, name: str, dtype, dev: int, shape):
    """_want for a tensor of any strides whose last dimension is contiguous; returns its strides."""
    strides = t.stride()
    if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or (strides[-1] != 1 and shape[-1] > 1):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return strides


# --------------------------------------------------------------- host queries

def taylor_attn_version() -> int:
    return int(lib().taylor_attn_version())


def taylor_attn_num_features(d_k: int, n: int) -> int:
    return int(lib().taylor_attn_num_features(d_k, n))


def taylor_attn_state_stride(d_k: int, d_v: int, n: int) -> int:
    return int(lib().taylor_attn_state_stride(d_k, d_v, n))


def taylor_attn_feature_index(d_k: int, n: int) -> Tuple[np.ndarray, np.ndarray]:
    """(deg [F], idx [F, max(n-1, 1)]) in host memory, -1 padded."""
    F = taylor_attn_num_features(d_k, n)
    if F < 0:
        raise TaylorAttnError(TAYLOR_ERR_UNSUPPORTED, "taylor_attn_feature_index")
    width = max(n - 1, 1)
    deg = np.empty(F, dtype=np.int32)
    idx = np.empty(F * width, dtype=np.int32)
    _check(lib().taylor_attn_feature_index(d_k, n, deg.ctypes.data, idx.ctypes.data),
           "taylor_attn_feature_index")
    return deg, idx.reshape(F, width)


# --------------------------------------------------------------- device calls

def taylor_attn_feature_map(x: torch.Tensor, n: int, tau: float = 1.0, query_side: bool = False,
                            phi: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """phi(x) for x [..., d_k] fp32 -> [..., F] fp32."""
    d_k = x.shape[-1]
    F = taylor_attn_num_features(d_k, n)
    if F < 0:
        raise TaylorAttnError(TAYLOR_ERR_UNSUPPORTED, "taylor_attn_feature_map")
    _need(x, "x", torch.float32)
    T = x.numel() // d_k if d_k else 0
    if phi is None:
        phi = torch.empty(x.shape[:-1] + (F,), dtype=torch.float32, device=x.device)
    _need(phi, "phi", torch.float32, x.device, x.shape[:-1] + (F,))
    _check(lib().taylor_attn_feature_map(_ptr(x), _ptr(phi), T, d_k, n, float(tau), int(bool(query_side)),
                                         _stream(stream)), "taylor_attn_feature_map")
    return phi


def _prefill(name, q, k, v, n, tau, out, state_out, stream):
    dtype = torch.bfloat16 if name == "taylor_attn_prefill" else torch.float32
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, H, N, d_k = q.shape
    d_v = v.shape[-1]
    _need(q, "q", dtype)
    _need(k, "k", dtype, q.device, (B, H, N, d_k))
    _need(v, "v", dtype, q.device, (B, H, N, d_v))
    if out is None:
        out = torch.empty((B, H, N, d_v), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, q.device, (B, H, N, d_v))
    if state_out is True:
        stride = taylor_attn_state_stride(d_k, d_v, n)
        if stride < 0:
            raise TaylorAttnError(TAYLOR_ERR_UNSUPPORTED, name)
        state_out = torch.empty((B, H, stride), dtype=torch.float32, device=q.device)
    if state_out is not None:
        _need(state_out, "state_out", torch.float32, q.device,
              (B, H, taylor_attn_state_stride(d_k, d_v, n)))
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(state_out), B, H, N, d_k,
                              d_v, n, float(tau), _stream(stream))
    _check(rc, name)
    return out, state_out


def taylor_attn_prefill(q, k, v, n: int, tau: float, out=None, state_out=None, stream=None):
    """bf16 q, k [B,H,N,d_k], v [B,H,N,d_v] -> (out fp32 [B,H,N,d_v], state or None).
    Pass ``state_out=True`` to have the final state allocated and returned."""
    return _prefill("taylor_attn_prefill", q, k, v, n, tau, out, state_out, stream)


def taylor_attn_prefill_f32(q, k, v, n: int, tau: float, out=None, state_out=None, stream=None):
    """taylor_attn_prefill with fp32 q, k, v."""
    return _prefill("taylor_attn_prefill_f32", q, k, v, n, tau, out, state_out, stream)


def _prefill_from_state(name, q, k, v, state_in, n, tau, out, state_out, stream):
    dtype = torch.bfloat16 if name == "taylor_attn_prefill_from_state" else torch.float32
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, H, N, d_k = q.shape
    d_v = v.shape[-1]
    stride = taylor_attn_state_stride(d_k, d_v, n)
    _need(q, "q", dtype)
    _need(k, "k", dtype, q.device, (B, H, N, d_k))
    _need(v, "v", dtype, q.device, (B, H, N, d_v))
    _need(state_in, "state_in", torch.float32, q.device, (B, H, stride))
    if out is None:
        out = torch.empty((B, H, N, d_v), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, q.device, (B, H, N, d_v))
    if state_out is True:
        state_out = torch.empty((B, H, stride), dtype=torch.float32, device=q.device)
    if state_out is not None:
        _need(state_out, "state_out", torch.float32, q.device, (B, H, stride))
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(state_in), _ptr(out), _ptr(state_out), B, H, N,
                              d_k, d_v, n, float(tau), _stream(stream))
    _check(rc, name)
    return out, state_out


def taylor_attn_prefill_from_state(q, k, v, state_in, n: int, tau: float, out=None, state_out=None,
                                   stream=None):
    """Prefill continuing from a carried state [B, H, stride]; bf16 q, k, v.
    ``state_out=True`` allocates the final state; it may also be ``state_in``."""
    return _prefill_from_state("taylor_attn_prefill_from_state", q, k, v, state_in, n, tau, out, state_out,
                               stream)


def taylor_attn_prefill_from_state_f32(q, k, v, state_in, n: int, tau: float, out=None, state_out=None,
                                       stream=None):
    return _prefill_from_state("taylor_attn_prefill_from_state_f32", q, k, v, state_in, n, tau, out, state_out,
                               stream)


def taylor_attn_prefill_f32_noalloc(q, k, v, n: int, tau: float, out=None, state_out=None, stream=None):
    """taylor_attn_prefill_f32 without any device allocation inside the call:
    its scratch is a fixed array in the library (see the header).  The caller
    passes every input and output; outputs are created here only when not
    given."""
    return _prefill("taylor_attn_prefill_f32_noalloc", q, k, v, n, tau, out, state_out, stream)


def taylor_attn_prefill_noalloc_scratch_floats() -> int:
    return int(lib().taylor_attn_prefill_noalloc_scratch_floats())


def _decode(name, q, k, v, state, n, tau, out, stream, order=None):
    dtype = torch.float32 if name.endswith("_f32") else torch.bfloat16
    if q.dim() != 3:
        raise ValueError("q, k must be [B, H, d_k] and v [B, H, d_v]")
    B, H, d_k = q.shape
    d_v = v.shape[-1]
    _need(q, "q", dtype)
    _need(k, "k", dtype, q.device, (B, H, d_k))
    _need(v, "v", dtype, q.device, (B, H, d_v))
    _need(state, "state", torch.float32, q.device, (B, H, taylor_attn_state_stride(d_k, d_v, n)))
    if out is None:
        out = torch.empty((B, H, d_v), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, q.device, (B, H, d_v))
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(state), _ptr(out), B, H, d_k, d_v,
                              n if order is None else order, float(tau), _stream(stream))
    _check(rc, name)
    return out


def taylor_attn_decode(q, k, v, state, n: int, tau: float, out=None, stream=None):
    """One token per (b, h): bf16 q, k [B,H,d_k], v [B,H,d_v]; ``state`` is
    updated in place; returns out fp32 [B,H,d_v]."""
    return _decode("taylor_attn_decode", q, k, v, state, n, tau, out, stream)


def taylor_attn_decode_f32(q, k, v, state, n: int, tau: float, out=None, stream=None):
    return _decode("taylor_attn_decode_f32", q, k, v, state, n, tau, out, stream)


def taylor_attn_centred_decode(q, k, v, state, order: int, tau: float, out=None, stream=None):
    """One token per (b, h) with the mean-centred softmax expansion of order
    1 or 2: bf16 q, k [B,H,d_k], v [B,H,d_v]; ``state`` is the n = 3 Taylor
    state [B,H,stride(d_k, d_v, 3)], updated in place; returns out fp32
    [B,H,d_v]."""
    return _decode("taylor_attn_centred_decode", q, k, v, state, 3, tau, out, stream, order=order)


def taylor_attn_centred_decode_f32(q, k, v, state, order: int, tau: float, out=None, stream=None):
    return _decode("taylor_attn_centred_decode_f32", q, k, v, state, 3, tau, out, stream, order=order)


def _centred_prefill(name, q, k, v, order, tau, out, state_out, stream):
    dtype = torch.bfloat16 if name == "taylor_attn_centred_prefill" else torch.float32
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    B, H, N, d_k = q.shape
    d_v = v.shape[-1]
    _need(q, "q", dtype)
    _need(k, "k", dtype, q.device, (B, H, N, d_k))
    _need(v, "v", dtype, q.device, (B, H, N, d_v))
    if out is None:
        out = torch.empty((B, H, N, d_v), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, q.device, (B, H, N, d_v))
    stride = taylor_attn_state_stride(d_k, d_v, 3)
    if state_out is True:
        if stride < 0:
            raise TaylorAttnError(TAYLOR_ERR_UNSUPPORTED, name)
        state_out = torch.empty((B, H, stride), dtype=torch.float32, device=q.device)
    if state_out is not None:
        _need(state_out, "state_out", torch.float32, q.device, (B, H, stride))
    rc = getattr(lib(), name)(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(state_out), B, H, N, d_k,
                              d_v, int(order), float(tau), _stream(stream))
    _check(rc, name)
    return out, state_out


def taylor_attn_centred_prefill(q, k, v, order: int, tau: float, out=None, state_out=None, stream=None):
    """Mean-centred softmax expansion (order 1 or 2), causal prefill: bf16 q,
    k [B,H,N,d_k], v [B,H,N,d_v] -> (out fp32, n = 3 Taylor state or None)."""
    return _centred_prefill("taylor_attn_centred_prefill", q, k, v, order, tau, out, state_out, stream)


def taylor_attn_centred_prefill_f32(q, k, v, order: int, tau: float, out=None, state_out=None, stream=None):
    """taylor_attn_centred_prefill with fp32 q, k, v."""
    return _centred_prefill("taylor_attn_centred_prefill_f32", q, k, v, order, tau, out, state_out, stream)


def taylor_attn_state_merge(a, b, d_k: int, d_v: int, n: int, out=None, stream=None):
    """a + b for states [B, H, stride] (out may be a or b)."""
    if a.dim() != 3:
        raise ValueError("states must be [B, H, stride]")
    B, H, stride = a.shape
    if stride != taylor_attn_state_stride(d_k, d_v, n):
        raise ValueError("state stride does not match (d_k, d_v, n)")
    _need(a, "a", torch.float32)
    _need(b, "b", torch.float32, a.device, a.shape)
    if out is None:
        out = torch.empty_like(a)
    _need(out, "out", torch.float32, a.device, a.shape)
    _check(lib().taylor_attn_state_merge(_ptr(a), _ptr(b), _ptr(out), B, H, d_k, d_v, n, _stream(stream)),
           "taylor_attn_state_merge")
    return out


# Host arrays of the calls (strides, frequencies) go as bytes, which ctypes
# passes by address; building a ctypes array takes five times as long.
_three = struct.Struct("3q").pack
_two = struct.Struct("2q").pack


def _qk_sides(q, k, freqs, positions, q_weight, k_weight, dtype):
    """Checks what both directions share: sizes, device, strides of q and k, frequencies."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k must be [B, N, H, d]")
    B, N, Hq, d = q.shape
    Hk, dev = k.size(2), q.get_device()
    qs = _rows(q, "q", dtype, dev, q.shape)
    ks = _rows(k, "k", dtype, dev, (B, N, Hk, d))
    if q_weight is not None:
        _want(q_weight, "q_weight", torch.float32, dev, (d,))
    if k_weight is not None:
        _want(k_weight, "k_weight", torch.float32, dev, (d,))
    if positions is not None:
        _want(positions, "positions", torch.int64, dev, (B, N))
    freqs = np.asarray(freqs, dtype=np.float64)
    if freqs.ndim != 1:
        raise ValueError("freqs must hold one frequency for each rotated pair")
    return B, N, Hq, Hk, d, dev, qs, ks, 2 * len(freqs), freqs.tobytes()


def _qk_norm_rope(name, dtype, q, k, freqs, positions, pos0, q_weight, k_weight, interleaved, eps, q_out, k_out,
                  stream):
    if _elsewhere(q, stream):
        with _on(q, stream):
            return _qk_norm_rope(name, dtype, q, k, freqs, positions, pos0, q_weight, k_weight, interleaved, eps,
                                 q_out, k_out, None)
    B, N, Hq, Hk, d, dev, qs, ks, rot, table = _qk_sides(q, k, freqs, positions, q_weight, k_weight, dtype)
    _fits(name, B, N, Hq, Hk, d, rot)
    if q_out is None:
        q_out = q.new_empty(B, Hq, N, d)
    else:
        _want(q_out, "q_out", dtype, dev, (B, Hq, N, d))
    if k_out is None:
        k_out = k.new_empty(B, Hk, N, d)
    else:
        _want(k_out, "k_out", dtype, dev, (B, Hk, N, d))
    rc = getattr(lib(), name)(q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions), pos0,
                              table, rot, bool(interleaved), q_out.data_ptr(),
                              k_out.data_ptr(), B, N, Hq, Hk, d, _three(*qs[:3]), _three(*ks[:3]), eps,
                              _current(dev))
    if rc:
        raise TaylorAttnError(rc, name)
    return q_out, k_out


def taylor_attn_qk_norm_rope(q, k, freqs, positions=None, pos0: int = 0, q_weight=None, k_weight=None,
                             interleaved: bool = False, eps: float = 0.0, q_out=None, k_out=None, stream=None):
    """Unit norms and position rotation of bf16 q [B,N,Hq,d], k [B,N,Hk,d]
    (any strides, last dimension contiguous) -> head-major q_out [B,Hq,N,d],
    k_out [B,Hk,N,d].  ``freqs`` holds the rot/2 frequencies on the host
    (rope_freqs); ``positions`` int64 [B,N], else pos0 + n."""
    return _qk_norm_rope("taylor_attn_qk_norm_rope", torch.bfloat16, q, k, freqs, positions, pos0, q_weight,
                         k_weight, interleaved, eps, q_out, k_out, stream)


def taylor_attn_qk_norm_rope_f32(q, k, freqs, positions=None, pos0: int = 0, q_weight=None, k_weight=None,
                                 interleaved: bool = False, eps: float = 0.0, q_out=None, k_out=None, stream=None):
    """taylor_attn_qk_norm_rope with fp32 tensors."""
    return _qk_norm_rope("taylor_attn_qk_norm_rope_f32", torch.float32, q, k, freqs, positions, pos0, q_weight,
                         k_weight, interleaved, eps, q_out, k_out, stream)


def _qk_norm_rope_backward(name, dtype, q, k, dq_out, dk_out, freqs, positions, pos0, q_weight, k_weight,
                           interleaved, eps, dq, dk, stream):
    if _elsewhere(q, stream):
        with _on(q, stream):
            return _qk_norm_rope_backward(name, dtype, q, k, dq_out, dk_out, freqs, positions, pos0, q_weight,
                                          k_weight, interleaved, eps, dq, dk, None)
    B, N, Hq, Hk, d, dev, qs, ks, rot, table = _qk_sides(q, k, freqs, positions, q_weight, k_weight, dtype)
    _fits(name, B, N, Hq, Hk, d, rot)
    _want(dq_out, "dq_out", dtype, dev, (B, Hq, N, d))
    _want(dk_out, "dk_out", dtype, dev, (B, Hk, N, d))
    if dq is None:
        dq, dqs = q.new_empty(B, N, Hq, d), (N * Hq * d, Hq * d, d)
    else:
        dqs = _rows(dq, "dq", dtype, dev, q.shape)
    if dk is None:
        dk, dks = k.new_empty(B, N, Hk, d), (N * Hk * d, Hk * d, d)
    else:
        dks = _rows(dk, "dk", dtype, dev, k.shape)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    rc = getattr(lib(), name)(q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), _ptr(q_weight),
                              _ptr(k_weight), _ptr(positions), pos0, table, rot,
                              bool(interleaved), dq.data_ptr(), dk.data_ptr(), _ptr(dqw), _ptr(dkw), B, N, Hq, Hk, d,
                              _three(*qs[:3]), _three(*ks[:3]), _three(*dqs[:3]), _three(*dks[:3]), eps,
                              _current(dev))
    if rc:
        raise TaylorAttnError(rc, name)
    return dq, dk, dqw, dkw


def taylor_attn_qk_norm_rope_backward(q, k, dq_out, dk_out, freqs, positions=None, pos0: int = 0, q_weight=None,
                                      k_weight=None, interleaved: bool = False, eps: float = 0.0, dq=None, dk=None,
                                      stream=None):
    """Gradients (dq [B,N,Hq,d], dk [B,N,Hk,d], dq_weight, dk_weight) of
    taylor_attn_qk_norm_rope from its inputs and dq_out [B,Hq,N,d], dk_out
    [B,Hk,N,d]; ``dq``, ``dk`` may be slices of a packed gradient.  A weight's
    gradient is None where there is no weight."""
    return _qk_norm_rope_backward("taylor_attn_qk_norm_rope_backward", torch.bfloat16, q, k, dq_out, dk_out, freqs,
                                  positions, pos0, q_weight, k_weight, interleaved, eps, dq, dk, stream)


def taylor_attn_qk_norm_rope_backward_f32(q, k, dq_out, dk_out, freqs, positions=None, pos0: int = 0, q_weight=None,
                                          k_weight=None, interleaved: bool = False, eps: float = 0.0, dq=None,
                                          dk=None, stream=None):
    """taylor_attn_qk_norm_rope_backward with fp32 tensors."""
    return _qk_norm_rope_backward("taylor_attn_qk_norm_rope_backward_f32", torch.float32, q, k, dq_out, dk_out,
                                  freqs, positions, pos0, q_weight, k_weight, interleaved, eps, dq, dk, stream)


def _gated_sides(gate, x, h0, lengths, dtype):
    if gate.dim() != 3:
        raise ValueError("gate, x must be [B, N, D]")
    B, N, D = shape = gate.shape
    dev = gate.get_device()
    gs = _rows(gate, "gate", dtype, dev, shape)
    xs = _rows(x, "x", dtype, dev, shape)
    if h0 is not None:
        _want(h0, "h0", torch.float32, dev, (B, D))
    if lengths is not None:
        _want(lengths, "lengths", torch.int32, dev, (B,))
    return B, N, D, dev, gs, xs


def _gated_scan(name, dtype, gate, x, coupled, h0, lengths, h, h_last, stream):
    if _elsewhere(gate, stream):
        with _on(gate, stream):
            return _gated_scan(name, dtype, gate, x, coupled, h0, lengths, h, h_last, None)
    B, N, D, dev, gs, xs = _gated_sides(gate, x, h0, lengths, dtype)
    _fits(name, B, N, D)
    if h is None:
        h = gate.new_empty(B, N, D)
    else:
        _want(h, "h", dtype, dev, (B, N, D))
    if h_last is True:
        h_last = torch.empty((B, D), dtype=torch.float32, device=gate.device) if h0 is None else torch.empty_like(h0)
    elif h_last is not None:
        _want(h_last, "h_last", torch.float32, dev, (B, D))
    rc = getattr(lib(), name)(gate.data_ptr(), x.data_ptr(), _ptr(h0), _ptr(lengths), h.data_ptr(), _ptr(h_last), B, N,
                              D, _two(*gs[:2]), _two(*xs[:2]), bool(coupled), _current(dev))
    if rc:
        raise TaylorAttnError(rc, name)
    return h, h_last


def taylor_attn_gated_scan(gate, x, coupled: bool = True, h0=None, lengths=None, h=None, h_last=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t (without
    ``coupled``: + x_t), a = sigmoid(gate), over bf16 gate, x [B,N,D] (any
    strides, last dimension contiguous) -> (h [B,N,D], last state fp32 [B,D]
    or None).  ``h_last=True`` has the last state allocated and returned; it
    may also be ``h0``.  ``lengths`` int32 [B]: rows past them give zeros."""
    return _gated_scan("taylor_attn_gated_scan", torch.bfloat16, gate, x, coupled, h0, lengths, h, h_last, stream)


def taylor_attn_gated_scan_f32(gate, x, coupled: bool = True, h0=None, lengths=None, h=None, h_last=None,
                               stream=None):
    """taylor_attn_gated_scan with fp32 tensors."""
    return _gated_scan("taylor_attn_gated_scan_f32", torch.float32, gate, x, coupled, h0, lengths, h, h_last, stream)


def _gated_scan_backward(name, dtype, gate, x, h, dh, coupled, h0, lengths, dh_last, dgate, dx, dh0, stream):
    if _elsewhere(gate, stream):
        with _on(gate, stream):
            return _gated_scan_backward(name, dtype, gate, x, h, dh, coupled, h0, lengths, dh_last, dgate, dx, dh0,
                                        None)
    B, N, D, dev, gs, xs = _gated_sides(gate, x, h0, lengths, dtype)
    _fits(name, B, N, D)
    _want(h, "h", dtype, dev, (B, N, D))
    _want(dh, "dh", dtype, dev, (B, N, D))
    if dh_last is not None:
        _want(dh_last, "dh_last", torch.float32, dev, (B, D))
    dgs = dxs = (N * D, D)
    if dgate is None:
        dgate = torch.empty_like(dh)
    else:
        dgs = _rows(dgate, "dgate", dtype, dev, gate.shape)
    if dx is None:
        dx = torch.empty_like(dh)
    else:
        dxs = _rows(dx, "dx", dtype, dev, gate.shape)
    if dh0 is True:
        dh0 = torch.empty((B, D), dtype=torch.float32, device=gate.device) if dh_last is None else torch.empty_like(dh_last)
    elif dh0 is False:
        dh0 = None
    elif dh0 is not None:
        _want(dh0, "dh0", torch.float32, dev, (B, D))
    rc = getattr(lib(), name)(gate.data_ptr(), x.data_ptr(), h.data_ptr(), dh.data_ptr(), _ptr(h0), _ptr(lengths),
                              _ptr(dh_last), dgate.data_ptr(), dx.data_ptr(), _ptr(dh0), B, N, D, _two(*gs[:2]),
                              _two(*xs[:2]), _two(*dgs[:2]), _two(*dxs[:2]), bool(coupled), _current(dev))
    if rc:
        raise TaylorAttnError(rc, name)
    return dgate, dx, dh0


def taylor_attn_gated_scan_backward(gate, x, h, dh, coupled: bool = True, h0=None, lengths=None, dh_last=None,
                                    dgate=None, dx=None, dh0=None, stream=None):
    """Gradients (dgate [B,N,D], dx [B,N,D], dh0 fp32 [B,D] or None) of
    taylor_attn_gated_scan from its inputs, its output h and the gradients dh
    [B,N,D], dh_last fp32 [B,D]; ``dgate``, ``dx`` may be slices of a packed
    gradient; ``dh0=True`` has the first state's gradient allocated."""
    return _gated_scan_backward("taylor_attn_gated_scan_backward", torch.bfloat16, gate, x, h, dh, coupled, h0,
                                lengths, dh_last, dgate, dx, dh0, stream)


def taylor_attn_gated_scan_backward_f32(gate, x, h, dh, coupled: bool = True, h0=None, lengths=None, dh_last=None,
                                        dgate=None, dx=None, dh0=None, stream=None):
    """taylor_attn_gated_scan_backward with fp32 tensors."""
    return _gated_scan_backward("taylor_attn_gated_scan_backward_f32", torch.float32, gate, x, h, dh, coupled, h0,
                                lengths, dh_last, dgate, dx, dh0, stream)


def _gated_step(name, dtype, gate, x, state, coupled, out, state_out, stream):
    if _elsewhere(gate, stream):
        with _on(gate, stream):
            return _gated_step(name, dtype, gate, x, state, coupled, out, state_out, None)
    if gate.dim() != 2:
        raise ValueError("gate, x must be [B, D]")
    B, D = shape = gate.shape
    _fits(name, B, D)
    dev = gate.get_device()
    gs = _rows(gate, "gate", dtype, dev, shape)
    xs = _rows(x, "x", dtype, dev, shape)
    _want(state, "state", torch.float32, dev, shape)
    if state_out is None:
        state_out = state
    else:
        _want(state_out, "state_out", torch.float32, dev, shape)
    if out is None:
        out = gate.new_empty(B, D)
    else:
        _want(out, "out", dtype, dev, shape)
    rc = getattr(lib(), name)(gate.data_ptr(), x.data_ptr(), state.data_ptr(), state_out.data_ptr(), out.data_ptr(), B,
                              D, gs[0], xs[0], bool(coupled), _current(dev))
    if rc:
        raise TaylorAttnError(rc, name)
    return out


def taylor_attn_gated_step(gate, x, state, coupled: bool = True, out=None, state_out=None, stream=None):
    """One token of the gated recurrence: bf16 gate, x [B,D] (rows of any
    stride), ``state`` fp32 [B,D] is updated in place unless ``state_out`` is
    given; returns out [B,D], the new state rounded."""
    return _gated_step("taylor_attn_gated_step", torch.bfloat16, gate, x, state, coupled, out, state_out, stream)


def taylor_attn_gated_step_f32(gate, x, state, coupled: bool = True, out=None, state_out=None, stream=None):
    """taylor_attn_gated_step with fp32 tensors."""
    return _gated_step("taylor_attn_gated_step_f32", torch.float32, gate, x, state, coupled, out, state_out, stream)


@functools.lru_cache(maxsize=256)
def _stride_of(d_k: int, d_v: int, n: int) -> int:
    return taylor_attn_state_stride(d_k, d_v, n)


def _shared_prefix_decode(name, dtype, q, k, v, prefix_state, k_cache, v_cache, lengths, n, tau, out, stream):
    if _elsewhere(q, stream):
        with _on(q, stream):
            return _shared_prefix_decode(name, dtype, q, k, v, prefix_state, k_cache, v_cache, lengths, n, tau, out,
                                         None)
    if q.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("q, k must be [B, H, d_k], v [B, H, d_v] and the caches [B, H, cap, d]")
    B, H, d_k = q.shape
    d_v, cap, dev = v.size(-1), k_cache.size(2), q.get_device()
    _fits(name, B, H, d_k, d_v, cap)
    stride = _stride_of(d_k, d_v, n)
    if stride < 0:
        raise TaylorAttnError(TAYLOR_ERR_UNSUPPORTED, name)
    _want(q, "q", dtype, dev, q.shape)
    _want(k, "k", dtype, dev, q.shape)
    _want(v, "v", dtype, dev, (B, H, d_v))
    _want(prefix_state, "prefix_state", torch.float32, dev, (1, H, stride) if prefix_state.dim() == 3 else (H, stride))
    _want(k_cache, "k_cache", dtype, dev, (B, H, cap, d_k))
    _want(v_cache, "v_cache", dtype, dev, (B, H, cap, d_v))
    _want(lengths, "lengths", torch.int32, dev, (B,))
    if out is None:
        out = prefix_state.new_empty(B, H, d_v)
    else:
        _want(out, "out", torch.float32, dev, (B, H, d_v))
    rc = getattr(lib(), name)(q.data_ptr(), k.data_ptr(), v.data_ptr(), prefix_state.data_ptr(), k_cache.data_ptr(),
                              v_cache.data_ptr(), lengths.data_ptr(), out.data_ptr(), B, H, cap, d_k, d_v, n, tau,
                              _current(dev))
    if rc:
        raise TaylorAttnError(rc, name)
    return out


def taylor_attn_shared_prefix_decode(q, k, v, prefix_state, k_cache, v_cache, lengths, n: int, tau: float, out=None,
                                     stream=None):
    """One token per sequence of a batch that shares a prefix: bf16 q, k
    [B,H,d_k], v [B,H,d_v]; ``prefix_state`` fp32 [H,stride] (or [1,H,stride],
    as a prefill returns it); the sequences' own tokens in ``k_cache``
    [B,H,cap,d_k], ``v_cache`` [B,H,cap,d_v], ``lengths`` int32 [B] of them.
    k and v are appended at row lengths[b]; returns out fp32 [B,H,d_v]."""
    return _shared_prefix_decode("taylor_attn_shared_prefix_decode", torch.bfloat16, q, k, v, prefix_state, k_cache,
                                 v_cache, lengths, n, tau, out, stream)


def taylor_attn_shared_prefix_decode_f32(q, k, v, prefix_state, k_cache, v_cache, lengths, n: int, tau: float,
                                         out=None, stream=None):
    """taylor_attn_shared_prefix_decode with fp32 q, k, v and caches."""
    return _shared_prefix_decode("taylor_attn_shared_prefix_decode_f32", torch.float32, q, k, v, prefix_state,
                                 k_cache, v_cache, lengths, n, tau, out, stream)


def taylor_attn_release_workspace() -> None:
    _check(lib().taylor_attn_release_workspace(), "taylor_attn_release_workspace")


def taylor_attn_selftest_bounded_wait(polls: int = 1000, stream=None) -> None:
    _check(lib().taylor_attn_selftest_bounded_wait(int(polls), _stream(stream)),
           "taylor_attn_selftest_bounded_wait")


def taylor_attn_device_errors(clear: bool = True) -> int:
    """Bits of the device error word (bounded waits that ran out); 0 if none."""
    flags = ctypes.c_uint(0)
    rc = lib().taylor_attn_device_errors(int(bool(clear)), ctypes.addressof(flags))
    if rc not in (TAYLOR_OK, TAYLOR_ERR_TIMEOUT):
        raise TaylorAttnError(rc, "taylor_attn_device_errors")
    return int(flags.value)


# --------------------------------------------------------------- kernel timing

def taylor_attn_timing_enable(on: bool) -> None:
    _check(lib().taylor_attn_timing_enable(int(bool(on))), "taylor_attn_timing_enable")


def taylor_attn_timing_read(max_kernels: int = 16):
    """{kernel name: (launches, total device ms)} since the last read."""
    names = ctypes.create_string_buffer(64 * max_kernels)
    launches = (ctypes.c_int * max_kernels)()
    ms = (ctypes.c_float * max_kernels)()
    rc = lib().taylor_attn_timing_read(max_kernels, ctypes.addressof(names), ctypes.addressof(launches),
                                       ctypes.addressof(ms))
    if rc < 0:
        raise TaylorAttnError(rc, "taylor_attn_timing_read")
    res = {}
    for i in range(min(rc, max_kernels)):
        nm = names.raw[64 * i:64 * i + 64].split(b"\0", 1)[0].decode()
        res[nm] = (int(launches[i]), float(ms[i]))
    return res


# --------------------------------------------------------------- layout helpers

def rope_freqs(rot: int, base: float = 10000.0) -> np.ndarray:
    """The rot/2 frequencies base^(-2j/rot) of a rotation, float64 on the host."""
    return float(base) ** (-np.arange(0, rot, 2) / max(rot, 1))


def state_view(state: torch.Tensor, d_k: int, d_v: int, n: int):
    """Views (S_v [..., F, d_v], z [..., F]) into a flat state [..., stride]."""
    F = taylor_attn_num_features(d_k, n)
    S_v = state[..., :F * d_v].unflatten(-1, (F, d_v))
    z = state[..., F * d_v:F * (d_v + 1)]
    return S_v, z


def state_logical(state: torch.Tensor, d_k: int, d_v: int, n: int) -> torch.Tensor:
    """Flat state [..., stride] -> [..., F, d_v + 1] with z as the last column."""
    S_v, z = state_view(state, d_k, d_v, n)
    return torch.cat([S_v, z.unsqueeze(-1)], dim=-1)


def state_flat(logical: torch.Tensor, d_k: int, d_v: int, n: int) -> torch.Tensor:
    """[..., F, d_v + 1] -> flat [..., stride] fp32 (zero padding), same device."""
    F = taylor_attn_num_features(d_k, n)
    stride = taylor_attn_state_stride(d_k, d_v, n)
    lead = logical.shape[:-2]
    flat = torch.zeros(lead + (stride,), dtype=torch.float32, device=logical.device)
    flat[..., :F * d_v] = logical[..., :d_v].reshape(lead + (F * d_v,)).float()
    flat[..., F * d_v:F * (d_v + 1)] = logical[..., d_v].float()
    return flat

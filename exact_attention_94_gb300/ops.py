"""PyTorch-facing wrappers of the C ABI (argument marshalling only).

Every function checks dtypes, devices, shapes and contiguity, allocates the
outputs with torch (PyTorch is the device-memory and stream provider here),
and calls the matching ``fa_*`` entry point on the current CUDA stream.  All
arithmetic happens in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib

_lib_handle = None


def lib():
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _lib.load()
    return _lib_handle


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_tensor_device(fn):
    """Runs a wrapper with the CUDA device of its tensors current (the library
    launches on the current device); tensors on two devices are refused."""
    @functools.wraps(fn)
    def wrapper(*args, **kwargs):
        tensors = [a for a in list(args) + list(kwargs.values()) if isinstance(a, torch.Tensor) and a.is_cuda]
        if not tensors:
            return fn(*args, **kwargs)
        dev = tensors[0].device
        if any(t.device != dev for t in tensors):
            raise ValueError("all CUDA tensors of a call must be on one device")
        with torch.cuda.device(dev):
            return fn(*args, **kwargs)
    return wrapper


def _check_bf16(name, t, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def set_option(opt: int, value: float) -> None:
    _lib.check(lib().fa_set_option(opt, float(value)), "fa_set_option")


def device_error() -> int:
    """Synchronises and returns the recorded device error code (0 = none)."""
    code = ctypes.c_uint(0)
    lib().fa_device_error(ctypes.byref(code))
    return int(code.value)


@_on_tensor_device
def fwd(q, k, v, causal: bool = False, scale: Optional[float] = None, out=None, lse=None,
        stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense forward.  q, k, v [B, N, H, d] bf16 -> (o [B, N, H, d], lse [B, H, N] fp32)."""
    _check_bf16("q", q)
    B, N, H, d = q.shape
    _check_bf16("k", k, q.shape)
    _check_bf16("v", v, q.shape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    l = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _check_bf16("out", o, q.shape)
    st = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, H, N, d, int(bool(causal)), scale,
                      _stream(stream))
    _lib.check(st, "fa_fwd")
    return o, l


@_on_tensor_device
def bwd(q, k, v, o, lse, dout, causal: bool = False, scale: Optional[float] = None, workspace=None,
        stream=None, out=None):
    """Dense backward -> (dq, dk, dv), each [B, N, H, d] bf16 (written into
    ``out`` = (dq, dk, dv) when given)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_bf16(name, t, q.shape)
    B, N, H, d = q.shape
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, H, N]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is not None:
        dq, dk, dv = out
        for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
            _check_bf16(name, t, q.shape)
    else:
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = lib().fa_bwd_workspace_bytes(B, H, N, d)
    ws = workspace if workspace is not None else torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace too small")
    st = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                      _ptr(ws), B, H, N, d, int(bool(causal)), scale, _stream(stream))
    _lib.check(st, "fa_bwd")
    return dq, dk, dv


def _check_cu(cu_seqlens, q):
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor")
    if cu_seqlens.device != q.device:
        raise ValueError("cu_seqlens must be on the device of q")


@_on_tensor_device
def fwd_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False, scale: Optional[float] = None,
               stream=None):
    """Packed forward.  q, k, v [total, H, d]; cu_seqlens int32 [S+1] on the device.
    Returns (o [total, H, d], lse [H, total])."""
    _check_bf16("q", q)
    total, H, d = q.shape
    _check_bf16("k", k, q.shape)
    _check_bf16("v", v, q.shape)
    _check_cu(cu_seqlens, q)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    l = torch.empty((H, total), dtype=torch.float32, device=q.device)
    st = lib().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), _ptr(cu_seqlens), cu_seqlens.numel() - 1,
                             int(max_seqlen), total, H, d, int(bool(causal)), scale, _stream(stream))
    _lib.check(st, "fa_fwd_varlen")
    return o, l


@_on_tensor_device
def bwd_varlen(q, k, v, o, lse, dout, cu_seqlens, max_seqlen: int, causal: bool = False,
               scale: Optional[float] = None, stream=None):
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_bf16(name, t, q.shape)
    total, H, d = q.shape
    _check_cu(cu_seqlens, q)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, total) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [H, total]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = lib().fa_bwd_varlen_workspace_bytes(total, H, d)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(ws), _ptr(cu_seqlens), cu_seqlens.numel() - 1, int(max_seqlen), total,
                             H, d, int(bool(causal)), scale, _stream(stream))
    _lib.check(st, "fa_bwd_varlen")
    return dq, dk, dv


@_on_tensor_device
def decode(q, k_cache, v_cache, num_splits: int = 0, scale: Optional[float] = None, stream=None,
           workspace=None):
    """Single-token decode.  q [B, 1, H, d]; caches [B, L, H, d].
    Returns (o [B, 1, H, d], lse [B, H])."""
    _check_bf16("q", q)
    B, one, H, d = q.shape
    if one != 1:
        raise ValueError("q must be [B, 1, H, d]")
    _check_bf16("k_cache", k_cache)
    L = k_cache.shape[1]
    if tuple(k_cache.shape) != (B, L, H, d):
        raise ValueError("k_cache must be [B, L, H, d]")
    _check_bf16("v_cache", v_cache, k_cache.shape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    splits = num_splits if num_splits > 0 else lib().fa_decode_num_splits(B, H, L, d)
    nbytes = lib().fa_decode_workspace_bytes(B, H, d, max(splits, 1))
    ws = workspace if workspace is not None else torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    l = torch.empty((B, H), dtype=torch.float32, device=q.device)
    st = lib().fa_decode_splitkv(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(l), B, H, L, d, splits,
                                 _ptr(ws), scale, _stream(stream))
    _lib.check(st, "fa_decode_splitkv")
    return o, l


@_on_tensor_device
def decode_paged(q, k_pages, v_pages, block_table, seq_lens, max_seq_len: int, num_splits: int = 0,
                 scale: Optional[float] = None, stream=None, workspace=None):
    """Single-token decode over a paged cache.  q [B, 1, H, d]; pages
    [num_pages, page_size, H, d]; block_table int32 [B, max_blocks] and
    seq_lens int32 [B] on the device.  Returns (o [B, 1, H, d], lse [B, H])."""
    _check_bf16("q", q)
    B, one, H, d = q.shape
    if one != 1:
        raise ValueError("q must be [B, 1, H, d]")
    _check_bf16("k_pages", k_pages)
    num_pages, page_size = k_pages.shape[0], k_pages.shape[1]
    if tuple(k_pages.shape) != (num_pages, page_size, H, d):
        raise ValueError("k_pages must be [num_pages, page_size, H, d]")
    _check_bf16("v_pages", v_pages, k_pages.shape)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if block_table.dim() != 2 or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
        raise ValueError("block_table must be [B, max_blocks] and seq_lens [B]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    splits = num_splits if num_splits > 0 else lib().fa_decode_num_splits(B, H, int(max_seq_len), d)
    nbytes = lib().fa_decode_workspace_bytes(B, H, d, max(splits, 1))
    ws = workspace if workspace is not None else torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    l = torch.empty((B, H), dtype=torch.float32, device=q.device)
    st = lib().fa_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seq_lens), _ptr(o),
                               _ptr(l), B, H, d, page_size, num_pages, block_table.shape[1], int(max_seq_len), splits,
                               _ptr(ws), scale, _stream(stream))
    _lib.check(st, "fa_decode_paged")
    return o, l


# ---------------------------------------------------------------- grouped-query attention

@_on_tensor_device
def fwd_gqa(q, k, v, causal: bool = False, scale: Optional[float] = None, stream=None):
    """q [B, N, Hq, d]; k, v [B, N, Hkv, d] with Hkv dividing Hq.
    Returns (o [B, N, Hq, d], lse [B, Hq, N])."""
    _check_bf16("q", q)
    B, N, Hq, d = q.shape
    _check_bf16("k", k)
    Hkv = k.shape[2]
    if tuple(k.shape) != (B, N, Hkv, d):
        raise ValueError("k must be [B, N, Hkv, d]")
    _check_bf16("v", v, k.shape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    l = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    st = lib().fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, Hq, Hkv, N, d, int(bool(causal)), scale,
                          _stream(stream))
    _lib.check(st, "fa_fwd_gqa")
    return o, l


@_on_tensor_device
def bwd_gqa(q, k, v, o, lse, dout, causal: bool = False, scale: Optional[float] = None, stream=None):
    """Gradients of fwd_gqa: (dq [B, N, Hq, d], dk, dv [B, N, Hkv, d])."""
    for name, t in (("q", q), ("o", o), ("dout", dout)):
        _check_bf16(name, t, q.shape)
    B, N, Hq, d = q.shape
    _check_bf16("k", k)
    Hkv = k.shape[2]
    _check_bf16("v", v, k.shape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = lib().fa_bwd_workspace_bytes(B, Hq, N, d)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                          _ptr(ws), B, Hq, Hkv, N, d, int(bool(causal)), scale, _stream(stream))
    _lib.check(st, "fa_bwd_gqa")
    return dq, dk, dv


@_on_tensor_device
def decode_gqa(q, k_cache, v_cache, num_splits: int = 0, scale: Optional[float] = None, stream=None):
    """q [B, 1, Hq, d]; caches [B, L, Hkv, d].  Returns (o [B, 1, Hq, d], lse [B, Hq])."""
    _check_bf16("q", q)
    B, one, Hq, d = q.shape
    _check_bf16("k_cache", k_cache)
    L, Hkv = k_cache.shape[1], k_cache.shape[2]
    if one != 1 or tuple(k_cache.shape) != (B, L, Hkv, d):
        raise ValueError("q must be [B, 1, Hq, d] and the caches [B, L, Hkv, d]")
    _check_bf16("v_cache", v_cache, k_cache.shape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    splits = num_splits if num_splits > 0 else lib().fa_decode_num_splits(B, Hkv, L, d)
    nbytes = lib().fa_decode_workspace_bytes(B, Hq, d, max(splits, 1))
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    l = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    st = lib().fa_decode_gqa(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(l), B, Hq, Hkv, L, d, splits,
                             _ptr(ws), scale, _stream(stream))
    _lib.check(st, "fa_decode_gqa")
    return o, l


# ---------------------------------------------------------------- masks: causal / sliding window, Nq != Nk

def _window(causal: bool, window: Optional[Tuple[int, int]]):
    """(window_left, window_right) of the C ABI; ``causal`` alone is (-1, 0)."""
    if window is None:
        return (-1, 0) if causal else (-1, -1)
    wl, wr = int(window[0]), int(window[1])
    if causal:
        wr = 0 if wr < 0 else min(wr, 0)
    return wl, wr


@_on_tensor_device
def fwd_masked(q, k, v, causal: bool = False, window: Optional[Tuple[int, int]] = None,
               scale: Optional[float] = None, stream=None):
    """q [B, Nq, Hq, d]; k, v [B, Nk, Hkv, d].  Bottom-right aligned mask:
    query i sees keys i + Nk - Nq - window[0] .. i + Nk - Nq + window[1]
    (-1 = open side; ``causal`` caps window[1] at 0).
    Returns (o [B, Nq, Hq, d], lse [B, Hq, Nq])."""
    _check_bf16("q", q)
    B, Nq, Hq, d = q.shape
    _check_bf16("k", k)
    Nk, Hkv = k.shape[1], k.shape[2]
    if tuple(k.shape) != (B, Nk, Hkv, d):
        raise ValueError("k must be [B, Nk, Hkv, d]")
    _check_bf16("v", v, k.shape)
    wl, wr = _window(causal, window)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    st = lib().fa_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), B, Hq, Hkv, Nq, Nk, d, wl, wr, scale,
                             _stream(stream))
    _lib.check(st, "fa_fwd_masked")
    return o, l


@_on_tensor_device
def bwd_masked(q, k, v, o, lse, dout, causal: bool = False, window: Optional[Tuple[int, int]] = None,
               scale: Optional[float] = None, stream=None):
    """Gradients of fwd_masked: (dq [B, Nq, Hq, d], dk, dv [B, Nk, Hkv, d])."""
    for name, t in (("q", q), ("o", o), ("dout", dout)):
        _check_bf16(name, t, q.shape)
    B, Nq, Hq, d = q.shape
    _check_bf16("k", k)
    Nk, Hkv = k.shape[1], k.shape[2]
    _check_bf16("v", v, k.shape)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Nq) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [B, Hq, Nq]")
    wl, wr = _window(causal, window)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = lib().fa_bwd_workspace_bytes(B, Hq, Nq, d)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(ws), B, Hq, Hkv, Nq, Nk, d, wl, wr, scale, _stream(stream))
    _lib.check(st, "fa_bwd_masked")
    return dq, dk, dv


@_on_tensor_device
def fwd_masked_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                      causal: bool = False, window: Optional[Tuple[int, int]] = None,
                      scale: Optional[float] = None, stream=None):
    """Packed fwd_masked: q [total_q, Hq, d]; k, v [total_k, Hkv, d]; int32
    offsets on the device.  Returns (o [total_q, Hq, d], lse [Hq, total_q])."""
    _check_bf16("q", q)
    total_q, Hq, d = q.shape
    _check_bf16("k", k)
    total_k, Hkv = k.shape[0], k.shape[1]
    if tuple(k.shape) != (total_k, Hkv, d):
        raise ValueError("k must be [total_k, Hkv, d]")
    _check_bf16("v", v, k.shape)
    _check_cu(cu_seqlens_q, q)
    _check_cu(cu_seqlens_k, q)
    if cu_seqlens_q.numel() != cu_seqlens_k.numel():
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    wl, wr = _window(causal, window)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    l = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    st = lib().fa_fwd_masked_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(l), _ptr(cu_seqlens_q),
                                    _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, int(max_seqlen_q),
                                    int(max_seqlen_k), total_q, total_k, Hq, Hkv, d, wl, wr, scale, _stream(stream))
    _lib.check(st, "fa_fwd_masked_varlen")
    return o, l


@_on_tensor_device
def bwd_masked_varlen(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, max_seqlen_k: int,
                      causal: bool = False, window: Optional[Tuple[int, int]] = None,
                      scale: Optional[float] = None, stream=None):
    """Gradients of fwd_masked_varlen: (dq [total_q, Hq, d], dk, dv [total_k, Hkv, d])."""
    for name, t in (("q", q), ("o", o), ("dout", dout)):
        _check_bf16(name, t, q.shape)
    total_q, Hq, d = q.shape
    _check_bf16("k", k)
    total_k, Hkv = k.shape[0], k.shape[1]
    _check_bf16("v", v, k.shape)
    _check_cu(cu_seqlens_q, q)
    _check_cu(cu_seqlens_k, q)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (Hq, total_q) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [Hq, total_q]")
    wl, wr = _window(causal, window)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = lib().fa_bwd_varlen_workspace_bytes(total_q, Hq, d)
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().fa_bwd_masked_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                                    _ptr(dv), _ptr(ws), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                    cu_seqlens_q.numel() - 1, int(max_seqlen_q), int(max_seqlen_k), total_q, total_k,
                                    Hq, Hkv, d, wl, wr, scale, _stream(stream))
    _lib.check(st, "fa_bwd_masked_varlen")
    return dq, dk, dv


# ---------------------------------------------------------------- FP8 forward

@_on_tensor_device
def fp8_quantize(x, signs=None, transpose: bool = False, stream=None):
    """e4m3 block quantisation of x [B, N, H, d] (bf16).  With ``signs`` (int8
    [d] of +-1 on the device) the rows are first rotated by the Hadamard matrix
    and the signs.  Returns (codes uint8 [B, N, H, d], or [B, H, d, n_pad] when
    transposed; scales fp32 [B, H, ceil(N / 128)])."""
    _check_bf16("x", x)
    B, N, H, d = x.shape
    nblk = (N + 127) // 128
    if signs is not None:
        if signs.dtype != torch.int8 or tuple(signs.shape) != (d,) or signs.device != x.device:
            raise ValueError("signs must be int8 [d] on the device of x")
    if transpose:
        codes = torch.empty((B, H, d, nblk * 128), dtype=torch.uint8, device=x.device)
    else:
        codes = torch.empty((B, N, H, d), dtype=torch.uint8, device=x.device)
    scales = torch.empty((B, H, nblk), dtype=torch.float32, device=x.device)
    st = lib().fa_fp8_quantize(_ptr(x), _ptr(signs), _ptr(codes), _ptr(scales), B, N, H, d,
                               int(signs is not None), int(bool(transpose)), _stream(stream))
    _lib.check(st, "fa_fp8_quantize")
    return codes, scales


@_on_tensor_device
def fwd_fp8_codes(q_codes, k_codes, vt_codes, q_scale, k_scale, v_scale, causal: bool = False,
                  window: Optional[Tuple[int, int]] = None, rotated: bool = True, scale: Optional[float] = None,
                  stream=None):
    """Attention on e4m3 operands from fp8_quantize (V transposed).
    Returns (o [B, Nq, Hq, d] bf16, lse [B, Hq, Nq])."""
    B, Nq, Hq, d = q_codes.shape
    Nk, Hkv = k_codes.shape[1], k_codes.shape[2]
    for name, t in (("q_codes", q_codes), ("k_codes", k_codes), ("vt_codes", vt_codes)):
        if t.dtype != torch.uint8 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor")
    if tuple(vt_codes.shape) != (B, Hkv, d, (Nk + 127) // 128 * 128):
        raise ValueError("vt_codes must be [B, Hkv, d, ceil(Nk / 128) * 128]")
    wl, wr = _window(causal, window)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty((B, Nq, Hq, d), dtype=torch.bfloat16, device=q_codes.device)
    l = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q_codes.device)
    st = lib().fa_fwd_fp8(_ptr(q_codes), _ptr(k_codes), _ptr(vt_codes), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale),
                          _ptr(o), _ptr(l), B, Hq, Hkv, Nq, Nk, d, wl, wr, int(bool(rotated)), scale,
                          _stream(stream))
    _lib.check(st, "fa_fwd_fp8")
    return o, l


@_on_tensor_device
def fwd_fp8(q, k, v, signs=None, causal: bool = False, window: Optional[Tuple[int, int]] = None,
            scale: Optional[float] = None, stream=None):
    """The FP8 forward from bf16 inputs: quantise Q and K (rotated when signs
    are given) and V (transposed), then attend.  Returns (o, lse)."""
    qc, qs = fp8_quantize(q, signs, stream=stream)
    kc, ks = fp8_quantize(k, signs, stream=stream)
    vc, vs = fp8_quantize(v, None, transpose=True, stream=stream)
    return fwd_fp8_codes(qc, kc, vc, qs, ks, vs, causal=causal, window=window, rotated=signs is not None,
                         scale=scale, stream=stream)


# ---------------------------------------------------------------- paged cache: write side

class PagePool:
    """Host page allocator of the C library (block tables, free list,
    reference counts); see fa_pool_* in fa.h.  Pages themselves are device
    tensors [num_pages, page_size, Hkv, d] that the caller owns."""

    def __init__(self, num_pages: int, page_size: int, max_seqs: int, max_blocks: int):
        self._lib = lib()
        self.handle = self._lib.fa_pool_create(num_pages, page_size, max_seqs, max_blocks)
        if not self.handle:
            raise _lib.FaError(_lib.FA_ERR_INVALID_ARG, "fa_pool_create")
        self.num_pages, self.page_size, self.max_seqs, self.max_blocks = num_pages, page_size, max_seqs, max_blocks

    def close(self):
        if self.handle:
            self._lib.fa_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()

    def free_pages(self) -> int:
        return self._lib.fa_pool_free_pages(self.handle)

    def refcount(self, page: int) -> int:
        return self._lib.fa_pool_refcount(self.handle, page)

    def add_seq(self) -> int:
        s = ctypes.c_int(-1)
        _lib.check(self._lib.fa_pool_add_seq(self.handle, ctypes.byref(s)), "fa_pool_add_seq")
        return s.value

    def fork(self, parent: int) -> int:
        s = ctypes.c_int(-1)
        _lib.check(self._lib.fa_pool_fork(self.handle, parent, ctypes.byref(s)), "fa_pool_fork")
        return s.value

    def release(self, seq: int) -> None:
        _lib.check(self._lib.fa_pool_release(self.handle, seq), "fa_pool_release")

    def reserve_append(self, seqs):
        """Next token of each sequence: int32 host tensors (page, slot, copy_src)."""
        seqs_t = torch.as_tensor(list(seqs), dtype=torch.int32)
        n = seqs_t.numel()
        page, slot, src = (torch.empty(n, dtype=torch.int32) for _ in range(3))
        _lib.check(self._lib.fa_pool_reserve_append(self.handle, _ptr(seqs_t), n, _ptr(page), _ptr(slot), _ptr(src)),
                   "fa_pool_reserve_append")
        return page, slot, src

    def export(self):
        """(block_table int32 [max_seqs, max_blocks], seq_lens int32 [max_seqs]), host."""
        table = torch.empty((self.max_seqs, self.max_blocks), dtype=torch.int32)
        lens = torch.empty(self.max_seqs, dtype=torch.int32)
        _lib.check(self._lib.fa_pool_export(self.handle, _ptr(table), _ptr(lens)), "fa_pool_export")
        return table, lens


@_on_tensor_device
def paged_append(k_new, v_new, k_pages, v_pages, page, slot, copy_src, stream=None):
    """Copies shared pages where copy_src >= 0, then writes each token's K, V
    rows ([n, Hkv, d] bf16) into (page, slot); index tensors int32 on the device."""
    _check_bf16("k_new", k_new)
    n, Hkv, d = k_new.shape
    _check_bf16("v_new", v_new, k_new.shape)
    _check_bf16("k_pages", k_pages)
    num_pages, P = k_pages.shape[0], k_pages.shape[1]
    if tuple(k_pages.shape) != (num_pages, P, Hkv, d):
        raise ValueError("k_pages must be [num_pages, page_size, Hkv, d]")
    _check_bf16("v_pages", v_pages, k_pages.shape)
    for name, t in (("page", page), ("slot", slot), ("copy_src", copy_src)):
        if t.dtype != torch.int32 or not t.is_cuda or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of {n} entries")
    st = lib().fa_paged_append(_ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages), _ptr(page), _ptr(slot),
                               _ptr(copy_src), n, Hkv, d, P, num_pages, _stream(stream))
    _lib.check(st, "fa_paged_append")


# ---------------------------------------------------------------- decode with a sliding window

def _window_span(L: int, window_left: int) -> int:
    return L if window_left < 0 or window_left >= L else window_left + 1


@_on_tensor_device
def decode_window(q, k_cache, v_cache, window_left: int, num_splits: int = 0, scale: Optional[float] = None,
                  stream=None):
    """Decode that sees only the last window_left + 1 keys of each cache.
    q [B, 1, Hq, d]; caches [B, L, Hkv, d].  Returns (o [B, 1, Hq, d], lse [B, Hq])."""
    _check_bf16("q", q)
    B, one, Hq, d = q.shape
    _check_bf16("k_cache", k_cache)
    L, Hkv = k_cache.shape[1], k_cache.shape[2]
    if one != 1 or tuple(k_cache.shape) != (B, L, Hkv, d):
        raise ValueError("q must be [B, 1, Hq, d] and the caches [B, L, Hkv, d]")
    _check_bf16("v_cache", v_cache, k_cache.shape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    span = _window_span(L, int(window_left))
    splits = num_splits if num_splits > 0 else lib().fa_decode_num_splits(B, Hkv, span, d)
    nbytes = lib().fa_decode_workspace_bytes(B, Hq, d, max(splits, 1))
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    l = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    st = lib().fa_decode_window(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(l), B, Hq, Hkv, L, d,
                                int(window_left), splits, _ptr(ws), scale, _stream(stream))
    _lib.check(st, "fa_decode_window")
    return o, l


@_on_tensor_device
def decode_paged_window(q, k_pages, v_pages, block_table, seq_lens, max_seq_len: int, window_left: int = -1,
                        num_splits: int = 0, scale: Optional[float] = None, stream=None):
    """Paged decode with grouped K/V heads and a sliding window.  q [B, 1, Hq, d];
    pages [num_pages, page_size, Hkv, d]; block_table int32 [B, max_blocks] and
    seq_lens int32 [B] on the device.  Returns (o [B, 1, Hq, d], lse [B, Hq])."""
    _check_bf16("q", q)
    B, one, Hq, d = q.shape
    if one != 1:
        raise ValueError("q must be [B, 1, Hq, d]")
    _check_bf16("k_pages", k_pages)
    num_pages, page_size, Hkv = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    if tuple(k_pages.shape) != (num_pages, page_size, Hkv, d):
        raise ValueError("k_pages must be [num_pages, page_size, Hkv, d]")
    _check_bf16("v_pages", v_pages, k_pages.shape)
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens)):
        if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if block_table.dim() != 2 or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
        raise ValueError("block_table must be [B, max_blocks] and seq_lens [B]")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    span = _window_span(int(max_seq_len), int(window_left))
    splits = num_splits if num_splits > 0 else lib().fa_decode_num_splits(B, Hkv, span, d)
    nbytes = lib().fa_decode_workspace_bytes(B, Hq, d, max(splits, 1))
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    l = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    st = lib().fa_decode_paged_window(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), _ptr(seq_lens),
                                      _ptr(o), _ptr(l), B, Hq, Hkv, d, page_size, num_pages, block_table.shape[1],
                                      int(max_seq_len), int(window_left), splits, _ptr(ws), scale, _stream(stream))
    _lib.check(st, "fa_decode_paged_window")
    return o, l


# ---------------------------------------------------------------- serving steps: planning, rotary, 8-bit cache
#
# A decode step launches a few kernels of some microseconds each, so these
# wrappers spend as little host time as their checks allow: one expression per
# tensor that holds for a good one, messages worked out only for a bad one,
# addresses passed as plain integers, the stream as its raw handle.

def _on_call_stream(fn):
    """Runs a wrapper with the device of its first CUDA tensor and the call's
    stream current: outputs and workspaces then come from that stream's own
    memory, so one call's cannot be handed to a call on another stream while it
    runs.  The wrapper gets the device's index and the stream's raw handle, and
    checks that every tensor is on that device."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kwargs):
        dev = -1
        for a in args:
            if isinstance(a, torch.Tensor):
                dev = a.get_device()
                if dev >= 0:
                    break
        if dev < 0:
            for a in kwargs.values():
                if isinstance(a, torch.Tensor) and a.is_cuda:
                    dev = a.get_device()
                    break
            else:
                return fn(*args, dev=-2, raw=0, **kwargs)  # nothing is on a GPU: refused by the checks
        if stream is not None:
            if stream.device.index != dev:
                raise ValueError("stream must be on the device of the tensors")
            with torch.cuda.stream(stream):
                return fn(*args, dev=dev, raw=stream.cuda_stream, **kwargs)
        if dev == torch._C._cuda_getDevice():  # (a tensor is there, so CUDA is set up)
            return fn(*args, dev=dev, raw=torch._C._cuda_getCurrentRawStream(dev), **kwargs)
        with torch.cuda.device(dev):
            return fn(*args, dev=dev, raw=torch._C._cuda_getCurrentRawStream(dev), **kwargs)
    return wrapper


def _refuse(name, t, dtype, dev, shape):
    """Says what is wrong with a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise (TypeError if dtype == torch.bfloat16 else ValueError)(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if t.get_device() != dev:
        raise ValueError("all CUDA tensors of a call must be on one device")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(name, t, dtype, dev, shape):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and t.is_contiguous()):
        _refuse(name, t, dtype, dev, shape)


def _check_dims(name, t, dtype, dev, dims, what):
    """As _check for a tensor that sets the call's sizes: its dimensions."""
    if isinstance(t, torch.Tensor):
        size = t.shape
        if len(size) != dims:
            raise ValueError(f"{name} must be {what}")
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
            return size
    _refuse(name, t, dtype, dev, None)


def _check_int(name, n):
    """A size as the C interface takes it (which would drop higher bits)."""
    n = int(n)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits")
    return n


def _check_rows(name, t, dev, shape=None):
    """A bf16 [..., H, d] tensor whose heads lie side by side and whose rows lie
    one stride apart (a slice of a fused projection, say).  Returns that stride."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.get_device() == dev
            and (shape is None or t.shape == shape)):
        _refuse(name, t, torch.bfloat16, dev, shape)
    size, step = t.shape, t.stride()
    if len(size) < 3:
        raise ValueError(f"{name} must be [..., H, d]")
    H, d = size[-2], size[-1]
    if len(size) == 3 and step[2] == 1 and step[1] == d and step[0] >= H * d:
        return step[0]
    if t.is_contiguous():
        return H * d
    rows = [(n, s) for n, s in zip(size[:-2], step[:-2]) if n != 1]
    ok = (d <= 1 or step[-1] == 1) and (H <= 1 or step[-2] == d)
    ok = ok and all(rows[i][1] == rows[i + 1][0] * rows[i + 1][1] for i in range(len(rows) - 1))
    if not ok or (rows and rows[-1][1] < H * d):
        raise ValueError(f"{name} must have contiguous heads and evenly spaced rows")
    return rows[-1][1] if rows else H * d


def _workspace(workspace, nbytes, dev, device):
    """The caller's workspace, checked, or one of the call's own."""
    if workspace is None:
        return torch.empty(max(16, nbytes), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of the other tensors")
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    return workspace


class PagePlan(NamedTuple):
    """What page_plan returns; int32 device tensors."""
    seq_lens: torch.Tensor    # [B] tokens of each request after the step
    cu_new: torch.Tensor      # [B + 1] packed offsets of the step's tokens
    page: torch.Tensor        # [max_tokens] where each row's token goes; -1 past the last
    slot: torch.Tensor        # [max_tokens]
    position: torch.Tensor    # [max_tokens] its position in its request; 0 past the last
    free_count: torch.Tensor  # [1] pages left


@_on_call_stream
def page_plan(ctx_lens, new_lens, free_pages, free_count, block_table, page_size: int, max_tokens: int, out=None, *,
              dev, raw) -> PagePlan:
    """Plans a step on the GPU.  ctx_lens, new_lens int32 [B]: tokens each
    request holds and gets; free_pages int32 [num_pages] and free_count int32
    [1]: the stack of free pages; block_table int32 [B, max_blocks], whose new
    entries are written.  No two requests may share a partly filled page (plan
    forks with PagePool); a finished request's pages go back by writing them
    behind the stack's top and raising free_count.  max_tokens: rows of the outputs, at least the step's
    tokens.  ``out``: a PagePlan to write into; its seq_lens may be ctx_lens and
    its free_count the given one, which advances them in place."""
    i32 = torch.int32
    B, max_blocks = _check_dims("block_table", block_table, i32, dev, 2, "[B, max_blocks]")
    (num_pages,) = _check_dims("free_pages", free_pages, i32, dev, 1, "[num_pages]")
    _check("ctx_lens", ctx_lens, i32, dev, (B,))
    _check("new_lens", new_lens, i32, dev, (B,))
    _check("free_count", free_count, i32, dev, (1,))
    n = _check_int("max_tokens", max_tokens)
    if n < 0:
        raise ValueError("max_tokens must not be negative")
    if out is None:  # one buffer, cut up
        buf = torch.empty(3 * n + 2 * B + 2, dtype=i32, device=block_table.device)
        page, slot, position, seq, cu, left = buf.split_with_sizes((n, n, n, B, B + 1, 1))
        out = PagePlan(seq, cu, page, slot, position, left)
    else:
        for name, t, size in zip(PagePlan._fields, out, (B, B + 1, n, n, n, 1)):
            _check(f"out.{name}", t, i32, dev, (size,))
    st = lib().fa_page_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(),
                            block_table.data_ptr(), *[t.data_ptr() for t in out], B, n, _check_int("page_size", page_size), num_pages,
                            max_blocks, raw)
    if st:
        _lib.check(st, "fa_page_plan")
    return out


class RopePlan:
    """Which axis each pair of a head turns with, and how fast; kept by the
    caller.  ``axis``: d / 2 integers, -1 for a pair that is copied; ``inv_freq``:
    d / 2 numbers, radians per position; ``neighbours``: pairs (2p, 2p + 1)
    instead of (p, p + d / 2); ``n_axes``: axes that positions have, 1 to 4, those
    that some pair turns with unless given."""

    def __init__(self, d: int, axis, inv_freq, neighbours: bool = False, n_axes: Optional[int] = None):
        axis, inv_freq = [int(a) for a in axis], [float(f) for f in inv_freq]
        if d not in (64, 128):
            raise _lib.FaError(_lib.FA_ERR_UNSUPPORTED, "RopePlan")
        if len(axis) != d // 2 or len(inv_freq) != d // 2:
            raise ValueError(f"axis and inv_freq must have {d // 2} entries")
        if any(not -1 <= a < 4 for a in axis) or not all(math.isfinite(f) for f in inv_freq):
            raise ValueError("axis entries must be -1 .. 3 and inv_freq finite")
        self.d, self.used_axes = d, max(1, max(axis) + 1)
        self.n_axes = self.used_axes if n_axes is None else int(n_axes)
        if not self.used_axes <= self.n_axes <= 4:
            raise ValueError(f"n_axes must be {self.used_axes} (the axes in use) to 4")
        self.struct = _lib.RopePlanStruct(self.n_axes, int(bool(neighbours)))
        self.struct.axis[:d // 2] = axis
        self.struct.inv_freq[:d // 2] = inv_freq
        self._ref = ctypes.byref(self.struct)


def rope_plan(d: int, sections, theta: float = 10000.0, per_axis: bool = False, neighbours: bool = False) -> RopePlan:
    """The usual plans.  ``sections``: pairs of each axis, in order, some of them
    none if need be; what they leave of the d / 2 pairs is copied.  Frequencies are theta^(-p / (d / 2)) of
    pair p (one ladder over the head, shared by the axes), or, per_axis, a
    ladder for each axis: theta^(-j / n) of pair j of its n."""
    sections = [int(n) for n in sections]
    if not sections or len(sections) > 4 or min(sections) < 0 or sum(sections) > d // 2:
        raise ValueError("sections must be 1 to 4 counts of pairs, d / 2 of them at most")
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    if per_axis:
        freq = [theta ** (-j / n) for n in sections for j in range(n)]
    else:
        freq = [theta ** (-p / (d // 2)) for p in range(len(axis))]
    rest = d // 2 - len(axis)
    return RopePlan(d, axis + [-1] * rest, freq + [0.0] * rest, neighbours, len(sections))


def _rope_side(name, t, o, plan, dev):
    """(rows, heads, address, address, stride, stride, output) of q or k."""
    stride = _check_rows(name, t, dev)
    size = t.shape
    H, d = size[-2], size[-1]
    if d != plan.d:
        raise ValueError(f"{name} has head dim {d}, the plan {plan.d}")
    if o is None:
        o, out_stride = torch.empty(size, dtype=torch.bfloat16, device=t.device), H * d
    else:
        out_stride = _check_rows(f"out {name}", o, dev, size)
    return t.numel() // max(1, H * d), H, t.data_ptr(), o.data_ptr(), stride, out_stride, o


def _plan_axes(plan, positions):
    """Axes that positions must have (last ones that no pair turns with may be left out)."""
    axes = plan.n_axes
    if plan.used_axes < axes and isinstance(positions, torch.Tensor) and positions.dim() == 2:
        axes = min(max(positions.shape[0], plan.used_axes), axes)
    return axes


def _rope(q, k, positions, plan, inverse, out, dev, raw):
    if not isinstance(plan, RopePlan):
        raise TypeError("plan must be a RopePlan")
    if q is None and k is None:
        raise ValueError("q or k must be given")
    oq, ok = out if out is not None else (None, None)
    none = (None, 0, None, None, 0, 0, None)
    nq, Hq, pq, poq, qs, qos, oq = _rope_side("q", q, oq, plan, dev) if q is not None else none
    nk, Hkv, pk, pok, ks, kos, ok = _rope_side("k", k, ok, plan, dev) if k is not None else none
    if nq is not None and nk is not None and nq != nk:
        raise ValueError("q and k must have the same rows")
    rows = nq if nq is not None else nk
    _check("positions", positions, torch.int32, dev, (_plan_axes(plan, positions), rows))
    st = lib().fa_rope_axes(pq, pk, poq, pok, positions.data_ptr(), plan._ref, rows, Hq, Hkv, plan.d, qs, ks, qos, kos,
                            inverse, raw)
    if st:
        _lib.check(st, "fa_rope_axes")
    return oq, ok


@_on_call_stream
def rope_axes(q, k, positions, plan: RopePlan, out=None, *, dev, raw):
    """Rotates q [..., Hq, d] and k [..., Hkv, d] (either may be None) by their
    rows' positions, int32 [plan.n_axes, rows]; last axes that no pair turns with
    may be left out of them.  Rows may lie a stride apart.
    Returns (q, k) rotated, in ``out`` = (q_out, k_out) when given (q_out may be q)."""
    return _rope(q, k, positions, plan, 0, out, dev, raw)


@_on_call_stream
def rope_axes_bwd(dq, dk, positions, plan: RopePlan, out=None, *, dev, raw):
    """Gradients of rope_axes: (dq, dk) with respect to what it was given, from
    those with respect to what it returned."""
    return _rope(dq, dk, positions, plan, 1, out, dev, raw)


def _check_kv8(k_codes, v_codes, k_scale, v_scale, dev):
    size = _check_dims("k_codes", k_codes, torch.uint8, dev, 4, "[num_pages, Hkv, page_size, d]")
    _check("v_codes", v_codes, torch.uint8, dev, size)
    _check("k_scale", k_scale, torch.float32, dev, size[:2])
    _check("v_scale", v_scale, torch.float32, dev, size[:2])
    return size


@_on_call_stream
def kv8_append(k_new, v_new, k_codes, v_codes, k_scale, v_scale, page, slot, copy_src=None, *, dev, raw) -> None:
    """Quantises tokens ([n, Hkv, d] bf16, rows may lie a stride apart) into the
    8-bit cache: codes uint8 [num_pages, Hkv, page_size, d] and scales fp32
    [num_pages, Hkv], updated.  page, slot (and copy_src) int32 [n] as from
    page_plan or PagePool.reserve_append; page -1 skips a row."""
    num_pages, Hkv, P, d = _check_kv8(k_codes, v_codes, k_scale, v_scale, dev)
    (n,) = _check_dims("page", page, torch.int32, dev, 1, "[n]")
    _check("slot", slot, torch.int32, dev, (n,))
    ks, vs = _check_rows("k_new", k_new, dev, (n, Hkv, d)), _check_rows("v_new", v_new, dev, (n, Hkv, d))
    if copy_src is not None:
        _check("copy_src", copy_src, torch.int32, dev, (n,))
        copy_src = copy_src.data_ptr()
    st = lib().fa_kv8_append(k_new.data_ptr(), v_new.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                             k_scale.data_ptr(), v_scale.data_ptr(), page.data_ptr(), slot.data_ptr(), copy_src, n, Hkv,
                             d, P, num_pages, ks, vs, raw)
    if st:
        _lib.check(st, "fa_kv8_append")


@functools.lru_cache(maxsize=1024)
def _kv8_shares(dev, B, Nq, Hq, Hkv, d, L, window_left, shares):
    """(shares, workspace bytes) of a call: they depend on its sizes and the device alone."""
    for name, n in (("max_seq_len", L), ("window_left", window_left), ("num_shares", shares)):
        _check_int(name, n)
    if shares == 0:
        shares = lib().fa_decode_kv8_num_shares(B, Nq, Hq, Hkv, L, window_left)
    return shares, max(16, lib().fa_decode_kv8_workspace_bytes(B, Nq, Hq, Hkv, d, max(shares, 1)))


@_on_call_stream
def decode_kv8(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, max_seq_len: int, window_left: int = -1,
               num_shares: int = 0, scale: Optional[float] = None, workspace=None, *, dev, raw):
    """Attention of q [B, Nq, Hq, d] over the 8-bit paged cache; query i of a
    request stands at seq_lens - Nq + i.  block_table int32 [B, max_blocks] and
    seq_lens int32 [B] on the device.  Returns (o [B, Nq, Hq, d], lse [B, Hq, Nq])."""
    num_pages, Hkv, P, d = _check_kv8(k_codes, v_codes, k_scale, v_scale, dev)
    B, Nq, Hq, dq = _check_dims("q", q, torch.bfloat16, dev, 4, f"[B, Nq, Hq, {d}]")
    if dq != d:
        raise ValueError(f"q must be [B, Nq, Hq, {d}]")
    rows, max_blocks = _check_dims("block_table", block_table, torch.int32, dev, 2, "[B, max_blocks]")
    if rows != B:
        raise ValueError(f"block_table has {rows} rows for {B} requests")
    _check("seq_lens", seq_lens, torch.int32, dev, (B,))
    L, wl = int(max_seq_len), int(window_left)
    shares, nbytes = _kv8_shares(dev, B, Nq, Hq, Hkv, d, L, wl, int(num_shares))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the device of q")
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    st = lib().fa_decode_kv8(q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                             v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                             lse.data_ptr(), B, Nq, Hq, Hkv, d, P, num_pages, max_blocks, L, wl, shares,
                             workspace.data_ptr(), 1.0 / math.sqrt(d) if scale is None else float(scale), raw)
    if st:
        _lib.check(st, "fa_decode_kv8")
    return o, lse


# ---------------------------------------------------------------- sampling steps: head norms with the rotation

def _norm_side(name, plan, dev, w, tensors, out):
    """(rows, heads, addresses, strides, output, weights are fp32) of q or k: the
    inputs `tensors`, of one shape, and the output."""
    x = tensors[0]
    strides = [_check_rows(name, x, dev)]
    size = x.shape
    H, d = size[-2], size[-1]
    if d != plan.d:
        raise ValueError(f"{name} has head dim {d}, the plan {plan.d}")
    strides += [_check_rows(f"dy{name}", t, dev, size) for t in tensors[1:]]
    wide = isinstance(w, torch.Tensor) and w.dtype is torch.float32
    _check(f"w{name}", w, torch.float32 if wide else torch.bfloat16, dev, (d,))
    if out is None:
        out = torch.empty(size, dtype=torch.bfloat16, device=x.device)
        strides.append(H * d)
    else:
        strides.append(_check_rows(f"out {name}", out, dev, size))
    return x.numel() // max(1, H * d), H, [t.data_ptr() for t in (*tensors, out)], strides, out, wide


def _norm_sides(qs, ks, wq, wk, positions, plan, out, dev):
    """Both sides' checks; an absent one has no addresses and no heads."""
    if not isinstance(plan, RopePlan):
        raise TypeError("plan must be a RopePlan")
    if qs[0] is None and ks[0] is None:
        raise ValueError("q or k must be given")
    oq, ok = out if out is not None else (None, None)
    n = len(qs) + 1
    none = (None, 0, [None] * n, [0] * n, None, None)
    q = _norm_side("q", plan, dev, wq, qs, oq) if qs[0] is not None else none
    k = _norm_side("k", plan, dev, wk, ks, ok) if ks[0] is not None else none
    if q[0] is not None and k[0] is not None and q[0] != k[0]:
        raise ValueError("q and k must have the same rows")
    if q[5] is not None and k[5] is not None and q[5] != k[5]:
        raise ValueError("wq and wk must have one dtype")
    rows = q[0] if q[0] is not None else k[0]
    _check("positions", positions, torch.int32, dev, (_plan_axes(plan, positions), rows))
    return q, k, rows, int(bool(q[5] or k[5]))


@_on_call_stream
def qk_norm_rope(q, k, wq, wk, positions, plan: RopePlan, eps: float = 1e-6, out=None, *, dev, raw):
    """Root-mean-square norms of the heads of q [..., Hq, d] and k [..., Hkv, d]
    (either may be None) with weights wq, wk [d] (bf16 or fp32), and their
    rotation as rope_axes does it, in one pass.  Returns (q, k), in ``out`` =
    (q_out, k_out) when given (q_out may be q)."""
    q, k, rows, wide = _norm_sides((q,), (k,), wq, wk, positions, plan, out, dev)
    st = lib().fa_qk_norm_rope(q[2][0], k[2][0], q[2][1], k[2][1], wq.data_ptr() if q[1] else None,
                               wk.data_ptr() if k[1] else None, positions.data_ptr(), plan._ref, rows, q[1], k[1], plan.d,
                               q[3][0], k[3][0], q[3][1], k[3][1], wide, float(eps), raw)
    if st:
        _lib.check(st, "fa_qk_norm_rope")
    return q[4], k[4]


@_on_call_stream
def qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, positions, plan: RopePlan, eps: float = 1e-6, out=None, workspace=None, *,
                     dev, raw):
    """Gradients of qk_norm_rope from those of what it returned: (dq, dk, dwq,
    dwk), the weights' in fp32; dq and dk in ``out`` when given (which may be dyq
    and dyk, or q and k)."""
    if (dyq is None) != (q is None) or (dyk is None) != (k is None):
        raise ValueError("q and dyq, k and dyk go together")
    q, k, rows, wide = _norm_sides((q, dyq), (k, dyk), wq, wk, positions, plan, out, dev)
    d = plan.d
    dwq, dwk = (torch.empty(d, dtype=torch.float32, device=positions.device) if x[1] else None for x in (q, k))
    workspace = _workspace(workspace, lib().fa_qk_norm_rope_bwd_workspace_bytes(rows, q[1], k[1], d), dev, positions.device)
    st = lib().fa_qk_norm_rope_bwd(q[2][1], k[2][1], q[2][0], k[2][0], q[2][2], k[2][2], wq.data_ptr() if q[1] else None,
                                   wk.data_ptr() if k[1] else None, dwq.data_ptr() if q[1] else None,
                                   dwk.data_ptr() if k[1] else None, positions.data_ptr(), plan._ref, rows, q[1], k[1], d,
                                   q[3][1], k[3][1], q[3][0], k[3][0], q[3][2], k[3][2], wide, float(eps),
                                   workspace.data_ptr(), raw)
    if st:
        _lib.check(st, "fa_qk_norm_rope_bwd")
    return q[4], k[4], dwq, dwk


# ---------------------------------------------------------------- sampling steps: attention of shared prefixes

@functools.lru_cache(maxsize=1024)
def _shared_bytes(dev, B, Nq, Hq, Hkv, d, groups, max_seq_len, window_left, shares):
    """Workspace bytes of a call: they depend on its sizes and the device alone."""
    for name, n in (("max_seq_len", max_seq_len), ("window_left", window_left), ("num_shares", shares)):
        _check_int(name, n)
    return lib().fa_decode_shared_workspace_bytes(B, Nq, Hq, Hkv, d, groups, shares)


def _shared_args(q, d, Hkv, block_table, seq_lens, group_starts, shared_lens, max_seq_len, window_left, num_shares, workspace,
                 dev):
    """Checks what both caches' calls take; (B, Nq, Hq, table's columns, groups, longest, window, shares, workspace, o, lse)."""
    B, Nq, Hq, dq = _check_dims("q", q, torch.bfloat16, dev, 4, f"[B, Nq, Hq, {d}]")
    if dq != d:
        raise ValueError(f"q must be [B, Nq, Hq, {d}]")
    rows, max_blocks = _check_dims("block_table", block_table, torch.int32, dev, 2, "[B, max_blocks]")
    if rows != B:
        raise ValueError(f"block_table has {rows} rows for {B} requests")
    (groups,) = _check_dims("shared_lens", shared_lens, torch.int32, dev, 1, "[groups]")
    _check("seq_lens", seq_lens, torch.int32, dev, (B,))
    _check("group_starts", group_starts, torch.int32, dev, (groups + 1,))
    L, wl, shares = int(max_seq_len), int(window_left), int(num_shares)
    device = q.device
    workspace = _workspace(workspace, _shared_bytes(dev, B, Nq, Hq, Hkv, d, groups, L, wl, shares), dev, device)
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=device)
    return B, Nq, Hq, max_blocks, groups, L, wl, shares, workspace, torch.empty_like(q), lse


@_on_call_stream
def decode_paged_shared(q, k_pages, v_pages, block_table, seq_lens, group_starts, shared_lens, max_seq_len: int,
                        window_left: int = -1, num_shares: int = 0, scale: Optional[float] = None, workspace=None, *, dev,
                        raw):
    """Attention of q [B, Nq, Hq, d] over pages [num_pages, page_size, Hkv, d],
    for requests in groups that share their first tokens, which are read once for
    all.  Requests group_starts[g] .. group_starts[g + 1] - 1 share shared_lens[g]
    tokens (int32 on the device; 0 for none); query i of a request stands at
    seq_lens - Nq + i.  Returns (o [B, Nq, Hq, d], lse [B, Hq, Nq])."""
    num_pages, P, Hkv, d = _check_dims("k_pages", k_pages, torch.bfloat16, dev, 4, "[num_pages, page_size, Hkv, d]")
    _check("v_pages", v_pages, torch.bfloat16, dev, k_pages.shape)
    B, Nq, Hq, blocks, groups, L, wl, shares, workspace, o, lse = _shared_args(
        q, d, Hkv, block_table, seq_lens, group_starts, shared_lens, max_seq_len, window_left, num_shares, workspace, dev)
    st = lib().fa_decode_paged_shared(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
                                      seq_lens.data_ptr(), group_starts.data_ptr(), shared_lens.data_ptr(), o.data_ptr(),
                                      lse.data_ptr(), B, Nq, Hq, Hkv, d, P, num_pages, blocks, L, groups, wl, shares,
                                      workspace.data_ptr(), 1.0 / math.sqrt(d) if scale is None else float(scale), raw)
    if st:
        _lib.check(st, "fa_decode_paged_shared")
    return o, lse


@_on_call_stream
def decode_kv8_shared(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, group_starts, shared_lens,
                      max_seq_len: int, window_left: int = -1, num_shares: int = 0, scale: Optional[float] = None,
                      workspace=None, *, dev, raw):
    """decode_paged_shared over the 8-bit paged cache (codes and scales as in
    decode_kv8).  Returns (o [B, Nq, Hq, d], lse [B, Hq, Nq])."""
    num_pages, Hkv, P, d = _check_kv8(k_codes, v_codes, k_scale, v_scale, dev)
    B, Nq, Hq, blocks, groups, L, wl, shares, workspace, o, lse = _shared_args(
        q, d, Hkv, block_table, seq_lens, group_starts, shared_lens, max_seq_len, window_left, num_shares, workspace, dev)
    st = lib().fa_decode_kv8_shared(q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                                    v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), group_starts.data_ptr(),
                                    shared_lens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Nq, Hq, Hkv, d, P, num_pages,
                                    blocks, L, groups, wl, shares, workspace.data_ptr(),
                                    1.0 / math.sqrt(d) if scale is None else float(scale), raw)
    if st:
        _lib.check(st, "fa_decode_kv8_shared")
    return o, lse

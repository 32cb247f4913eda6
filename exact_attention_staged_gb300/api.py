"""Python binding of libfa.so: argument marshalling only (ctypes).

Every step of the attention path runs in the library's CUDA kernels; PyTorch supplies device
memory and the current stream.  There is no fallback: when libfa.so is missing or the device
is not an sm_103 GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading
from typing import Optional, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")

FA_FP16, FA_BF16 = 0, 1
FA_OK, FA_ERR_INVALID, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = 0, -1, -2, -3, -4
FA_ERR_INTERNAL, FA_ERR_INDEX = -5, -6
FA_ROPE_PLAIN, FA_ROPE_LINEAR, FA_ROPE_NTK, FA_ROPE_BY_PARTS, FA_ROPE_BANDS = 0, 1, 2, 3, 4
FA_NOALLOC_MAX_ROWS = 1 << 20  # B*H*N limit of fa_bwd_noalloc

# exported names and their signatures, in the order include/fa.h declares them
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_u64, _f64 = ctypes.c_ulonglong, ctypes.c_double
SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa_fwd_blocksparse": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "fa_fwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "fa_fwd_fp8_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fa_fwd_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _f, _f, _i, _vp,
                        _vp, _sz, _vp]),
    "fa_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _i,
                    _f, _i, _vp, _vp]),
    "fa_bwd_gqa_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fa_bwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i,
                        _i, _i, _f, _i, _vp, _vp]),
    "fa_fwd_dropout": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _f,
                            _u64, _u64, _vp]),
    "fa_bwd_dropout": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i,
                            _i, _i, _f, _i, _vp, _f, _u64, _u64, _vp]),
    "fa_bwd_preprocess": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "fa_bwd_dkdv": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                         _vp, _vp]),
    "fa_bwd_dq": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "fa_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                            _f, _i, _vp, _vp]),
    "fa_decode_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp,
                       _sz, _vp]),
    "fa_rope_frequencies": (_i, [_vp, _vp, _i, _f64, _i, _f64, _f64, _f64, _f64]),
    "fa_rope": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                     _vp]),
    "fa_paged_check": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i]),
    "fa_paged_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
                             _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp]),
    "fa_paged_attn_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i, _i]),
    "fa_paged_attn": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                           _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa_sync_status": (_i, [_vp]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_debug_paged_pieces": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp, _i]),
    "fa_debug_set_visit_log": (_i, [_vp, _sz]),
    "fa_debug_set_wait_limit_ns": (_i, [ctypes.c_ulonglong]),
    "fa_debug_set_fault": (_i, [_i]),
    "fa_debug_set_dkdv_splits": (_i, [_i]),
}

_lib = None
_lock = threading.Lock()


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


def load(path: str = LIB_PATH):
    """Load libfa.so (built by ``exact_attention_staged_gb300.build``); raise if absent."""
    global _lib
    lib = _lib
    if lib is not None:  # loaded: no lock on the per-call path
        return lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m exact_attention_staged_gb300.build`")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().fa_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != FA_OK:
        raise FAError(code, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float16")


def _dev(t: Optional[torch.Tensor], name: str, like: Optional[torch.Tensor] = None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name} must match q in shape and dtype")
    return t.data_ptr()  # ctypes passes the int as the c_void_p argument


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream: Optional[torch.cuda.Stream], like: Optional[torch.Tensor] = None) -> int:
    """The CUDA stream handle to launch on: `stream`, else the current stream of the tensor's
    device (read as a raw handle: no Stream object is built on the per-call path)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and like is not None:
        return _raw_stream(like.device.index)
    return torch.cuda.current_stream().cuda_stream


def _shape(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("q, k, v must be [B, H, N, d]")
    return tuple(int(x) for x in q.shape)


def fwd(q, k, v, scale: Optional[float] = None, causal: bool = False, block_mask=None,
        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
        stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O, LSE = attention forward (fa_fwd, or fa_fwd_blocksparse when block_mask is given)."""
    lib = load()
    B, H, N, d = _shape(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be fp32 [B, H, N]")
    args = [_dev(q, "q"), _dev(k, "k", q), _dev(v, "v", q), _dev(out, "out", q), _dev(lse, "lse"),
            B, H, N, d, _dtype_code(q), float(scale), int(bool(causal))]
    if block_mask is None:
        _check(lib.fa_fwd(*args, _stream(stream, q)), "fa_fwd")
    else:
        if block_mask.dtype != torch.uint8:
            raise TypeError("block_mask must be uint8")
        _check(lib.fa_fwd_blocksparse(*args, _dev(block_mask, "block_mask"), _stream(stream, q)),
               "fa_fwd_blocksparse")
    return out, lse


def workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_bytes(B, H, N, d))


def bwd(q, k, v, o, lse, dout, scale: Optional[float] = None, causal: bool = False,
        block_mask=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV = attention backward (fa_bwd)."""
    lib = load()
    B, H, N, d = _shape(q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    nbytes = workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(lib.fa_bwd(_dev(q, "q"), _dev(k, "k", q), _dev(v, "v", q), _dev(o, "o", q),
                      _dev(dout, "dout", q), _dev(lse, "lse"), _dev(dq, "dq", q),
                      _dev(dk, "dk", q), _dev(dv, "dv", q), _dev(workspace, "workspace"),
                      nbytes, B, H, N, d, _dtype_code(q), float(scale), int(bool(causal)),
                      mask_ptr, _stream(stream, q)), "fa_bwd")
    return dq, dk, dv


def bwd_preprocess(o, dout, delta, stream=None):
    B, H, N, d = _shape(o)
    _check(load().fa_bwd_preprocess(_dev(o, "o"), _dev(dout, "dout", o), _dev(delta, "delta"),
                                    B, H, N, d, _dtype_code(o), _stream(stream, o)),
           "fa_bwd_preprocess")
    return delta


def bwd_dkdv(q, k, v, dout, lse, delta, dk, dv, scale=None, causal=False, block_mask=None,
             stream=None):
    B, H, N, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(load().fa_bwd_dkdv(_dev(q, "q"), _dev(k, "k", q), _dev(v, "v", q),
                              _dev(dout, "dout", q), _dev(lse, "lse"), _dev(delta, "delta"),
                              _dev(dk, "dk", q), _dev(dv, "dv", q), B, H, N, d, _dtype_code(q),
                              float(scale), int(bool(causal)), mask_ptr, _stream(stream, q)),
           "fa_bwd_dkdv")
    return dk, dv


def bwd_dq(q, k, v, dout, lse, delta, dq, scale=None, causal=False, block_mask=None,
           stream=None):
    B, H, N, d = _shape(q)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(load().fa_bwd_dq(_dev(q, "q"), _dev(k, "k", q), _dev(v, "v", q),
                            _dev(dout, "dout", q), _dev(lse, "lse"), _dev(delta, "delta"),
                            _dev(dq, "dq", q), B, H, N, d, _dtype_code(q), float(scale),
                            int(bool(causal)), mask_ptr, _stream(stream, q)), "fa_bwd_dq")
    return dq


def _kv_check(q, k, v):
    """K, V of grouped-query attention: [B, H_kv, N, d] with H_kv dividing H; returns H_kv."""
    B, H, N, d = _shape(q)
    for name, t in (("k", k), ("v", v)):
        if t.dim() != 4 or t.dtype != q.dtype or t.shape[0] != B or t.shape[2:] != q.shape[2:]:
            raise ValueError(f"{name} must be [B, H_kv, N, d] with the dtype of q")
    if k.shape != v.shape:
        raise ValueError("k and v must have the same shape")
    return int(k.shape[1])


def fwd_gqa(q, k, v, scale: Optional[float] = None, causal: bool = False, block_mask=None,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O, LSE = grouped-query attention forward (fa_fwd_gqa): k, v are [B, H_kv, N, d]."""
    lib = load()
    B, H, N, d = _shape(q)
    Hkv = _kv_check(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be fp32 [B, H, N]")
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(lib.fa_fwd_gqa(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", q),
                          _dev(lse, "lse"), B, H, Hkv, N, d, _dtype_code(q), float(scale),
                          int(bool(causal)), mask_ptr, _stream(stream, q)), "fa_fwd_gqa")
    return out, lse


def fp8_workspace_bytes(B: int, H_kv: int, N: int, d: int) -> int:
    return int(load().fa_fwd_fp8_workspace_bytes(B, H_kv, N, d))


def fwd_fp8(q, k, v, descale_q: float, descale_k: float, descale_v: float,
            scale: Optional[float] = None, causal: bool = False, block_mask=None, out=None,
            lse=None, workspace=None, stream=None):
    """O (bf16), LSE of attention on e4m3 codes (uint8 tensors) with per-tensor scales
    (fa_fwd_fp8): q [B, H, N, d], k, v [B, H_kv, N, d]."""
    lib = load()
    B, H, N, d = _shape(q)
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype != torch.uint8:
            raise TypeError(f"{name} must hold e4m3 codes as torch.uint8")
    if k.dim() != 4 or k.shape != v.shape or k.shape[0] != B or k.shape[2:] != q.shape[2:]:
        raise ValueError("k and v must be [B, H_kv, N, d]")
    Hkv = int(k.shape[1])
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q.device) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    nbytes = fp8_workspace_bytes(B, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=q.device)
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(lib.fa_fwd_fp8(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out"),
                          _dev(lse, "lse"), B, H, Hkv, N, d, float(scale), float(descale_q),
                          float(descale_k), float(descale_v), int(bool(causal)), mask_ptr,
                          _dev(workspace, "workspace"),
                          workspace.numel() * workspace.element_size(), _stream(stream, q)),
           "fa_fwd_fp8")
    return out, lse


def gqa_workspace_bytes(B: int, H: int, H_kv: int, N: int, d: int) -> int:
    return int(load().fa_bwd_gqa_workspace_bytes(B, H, H_kv, N, d))


def bwd_gqa(q, k, v, o, lse, dout, scale: Optional[float] = None, causal: bool = False,
            block_mask=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV = grouped-query attention backward (fa_bwd_gqa); dk, dv are [B, H_kv, N, d]."""
    lib = load()
    B, H, N, d = _shape(q)
    Hkv = _kv_check(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = gqa_workspace_bytes(B, H, Hkv, N, d)
    if nbytes == 0:
        raise ValueError("invalid grouped-query sizes")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(lib.fa_bwd_gqa(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o", q),
                          _dev(dout, "dout", q), _dev(lse, "lse"), _dev(dq, "dq", q),
                          _dev(dk, "dk", k), _dev(dv, "dv", k), _dev(workspace, "workspace"),
                          nbytes, B, H, Hkv, N, d, _dtype_code(q), float(scale),
                          int(bool(causal)), mask_ptr, _stream(stream, q)), "fa_bwd_gqa")
    return dq, dk, dv


def decode_workspace_bytes(B: int, H: int, H_kv: int, Nq: int, Nk: int, d: int) -> int:
    return int(load().fa_decode_workspace_bytes(B, H, H_kv, Nq, Nk, d))


def decode(q, k, v, scale: Optional[float] = None, causal: bool = False, kv_len=None,
           out=None, lse=None, workspace=None, stream=None):
    """O, LSE of Nq new rows q [B, H, Nq, d] against the cache k, v [B, H_kv, Nk, d] (fa_decode).

    kv_len: int32 CUDA tensor [B] of valid cache lengths, or None for Nk.
    """
    lib = load()
    B, H, Nq, d = _shape(q)
    if k.dim() != 4 or k.shape != v.shape or k.shape[0] != B or k.shape[3] != d \
            or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must be [B, H_kv, Nk, d] with the dtype of q")
    Hkv, Nk = int(k.shape[1]), int(k.shape[2])
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Nq):
        raise ValueError("lse must be fp32 [B, H, Nq]")
    if kv_len is not None and (kv_len.dtype != torch.int32 or tuple(kv_len.shape) != (B,)):
        raise ValueError("kv_len must be int32 [B]")
    nbytes = decode_workspace_bytes(B, H, Hkv, Nq, Nk, d)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    ws = None if workspace is None else _dev(workspace, "workspace")
    _check(lib.fa_decode(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", q),
                         _dev(lse, "lse"), None if kv_len is None else _dev(kv_len, "kv_len"),
                         B, H, Hkv, Nq, Nk, d, _dtype_code(q), float(scale), int(bool(causal)),
                         ws, nbytes, _stream(stream, q)), "fa_decode")
    return out, lse


def fwd_dropout(q, k, v, p_drop: float, seed: int, offset: int = 0,
                scale: Optional[float] = None, causal: bool = False, block_mask=None, out=None,
                lse=None, stream=None):
    """O, LSE with dropout on the probabilities (fa_fwd_dropout); k, v may have H_kv heads."""
    lib = load()
    B, H, N, d = _shape(q)
    Hkv = _kv_check(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(lib.fa_fwd_dropout(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(out, "out", q),
                              _dev(lse, "lse"), B, H, Hkv, N, d, _dtype_code(q), float(scale),
                              int(bool(causal)), mask_ptr, float(p_drop), int(seed), int(offset),
                              _stream(stream, q)), "fa_fwd_dropout")
    return out, lse


def bwd_dropout(q, k, v, o, lse, dout, p_drop: float, seed: int, offset: int = 0,
                scale: Optional[float] = None, causal: bool = False, block_mask=None, dq=None,
                dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of the forward with dropout (fa_bwd_dropout), same dropout arguments."""
    lib = load()
    B, H, N, d = _shape(q)
    Hkv = _kv_check(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = gqa_workspace_bytes(B, H, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    mask_ptr = None if block_mask is None else _dev(block_mask, "block_mask")
    _check(lib.fa_bwd_dropout(_dev(q, "q"), _dev(k, "k"), _dev(v, "v"), _dev(o, "o", q),
                              _dev(dout, "dout", q), _dev(lse, "lse"), _dev(dq, "dq", q),
                              _dev(dk, "dk", k), _dev(dv, "dv", k), _dev(workspace, "workspace"),
                              nbytes, B, H, Hkv, N, d, _dtype_code(q), float(scale),
                              int(bool(causal)), mask_ptr, float(p_drop), int(seed), int(offset),
                              _stream(stream, q)), "fa_bwd_dropout")
    return dq, dk, dv


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device
_DTYPES = {torch.bfloat16: FA_BF16, torch.float16: FA_FP16}
_I32, _I64, _F32, _U8 = torch.int32, torch.int64, torch.float32, torch.uint8
_empty = torch.empty
# strides are handed over as the bytes of a long long array
_pack10, _pack12, _pack14 = (struct.Struct(f"={n}q").pack for n in (10, 12, 14))


def _elsewhere(call, stream, device, tensors):
    """call() with `device` current and its launches and allocations on `stream`.  Tensors that
    belong to other streams are marked as used on it, so that their memory is not handed out
    again while the call's work may still read it."""
    if stream is not None and stream.device != device:
        raise ValueError("stream must belong to the tensors' device")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        result = call()
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
    return result


def _raw(dev: int) -> int:
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _check_place(dev: int, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name} must be a CUDA tensor on the same device as the others")


def _check_i32(t, name, shape):
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)}")


def _freq_table(freq) -> int:
    """Checks a frequency table; the number of rotated elements."""
    if freq.dtype is not _I64 or freq.dim() != 1 or not freq.is_contiguous():
        raise ValueError("freq must be a contiguous int64 table of rope_frequencies()")
    return 2 * freq.shape[0]


_SCALINGS = {"plain": FA_ROPE_PLAIN, "linear": FA_ROPE_LINEAR, "ntk": FA_ROPE_NTK,
             "by_parts": FA_ROPE_BY_PARTS, "bands": FA_ROPE_BANDS}


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain",
                     factor: float = 1.0, original_len: float = 0.0, low: float = 0.0,
                     high: float = 0.0, device=None) -> Tuple[torch.Tensor, float]:
    """The frequency table of rotary positions and its mscale (fa_rope_frequencies).

    The table (int64 bits of turns per position in units of 2^-64) is laid out once and passed to
    rope, rope_bwd and paged_append.  scaling: "plain", "linear", "ntk", "by_parts" or "bands";
    factor, original_len, low and high as its formula wants them.
    """
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    table = torch.empty(max(rot_dim // 2, 0), dtype=torch.int64)
    mscale = ctypes.c_float()
    _check(load().fa_rope_frequencies(table.data_ptr() or None, ctypes.addressof(mscale), rot_dim,
                                      base, _SCALINGS[scaling], factor, original_len, low, high),
           "fa_rope_frequencies")
    return table.to(device) if device is not None else table, float(mscale.value)


def _rope(q, k, freq, positions, interleaved, mscale, out_q, out_k, inverse, stream):
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    if stream is not None or dev != _current_device():
        return _elsewhere(lambda: _rope(q, k, freq, positions, interleaved, mscale, out_q, out_k,
                                        inverse, None),
                          stream, q.device, (q, k, freq, positions, out_q, out_k))
    if freq.get_device() != dev or positions is not None or out_q is not None \
            or out_k is not None or k is not None:
        _check_place(dev, k=k, freq=freq, positions=positions, out_q=out_q, out_k=out_k)
    shape, dt = q.shape, q.dtype
    code = _DTYPES.get(dt)
    if code is None:
        _dtype_code(q)
    if len(shape) != 4:
        raise ValueError("q, k must be [B, heads, N, d]")
    B, H, N, d = shape
    if positions is not None:
        _check_i32(positions, "positions", (B, N))
    if out_q is None:
        out_q = _empty(shape, dtype=dt, device=q.device)
    elif out_q.shape != shape or out_q.dtype is not dt:
        raise ValueError("out_q must match q in shape and dtype")
    a0, a1, a2, ae = q.stride()
    b0, b1, b2, be = out_q.stride()
    if k is None:
        if out_k is not None:
            raise ValueError("out_k needs k")
        Hkv = kp = kop = c0 = c1 = c2 = e0 = e1 = e2 = 0
        ce = ee = 1
    else:
        kshape = k.shape
        if len(kshape) != 4 or kshape[0] != B or kshape[2] != N or kshape[3] != d \
                or k.dtype is not dt:
            raise ValueError("k must be [B, H_kv, N, d] with the dtype of q")
        Hkv = kshape[1]
        if out_k is None:
            out_k = _empty(kshape, dtype=dt, device=q.device)
        elif out_k.shape != kshape or out_k.dtype is not dt:
            raise ValueError("out_k must match k in shape and dtype")
        c0, c1, c2, ce = k.stride()
        e0, e1, e2, ee = out_k.stride()
        kp, kop = k.data_ptr(), out_k.data_ptr()
    if ae != 1 or be != 1 or ce != 1 or ee != 1:
        raise ValueError("the rows of q, k and the outputs must be contiguous")
    rc = load().fa_rope(q.data_ptr(), out_q.data_ptr(), kp or None, kop or None,
                        _pack12(a0, a1, a2, b0, b1, b2, c0, c1, c2, e0, e1, e2), freq.data_ptr(),
                        None if positions is None else positions.data_ptr(), B, H, Hkv, N, d,
                        _freq_table(freq), code, 1 if interleaved else 0, inverse, mscale, _raw(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_rope")
    return out_q if k is None else (out_q, out_k)


def rope(q, k, freq, positions=None, interleaved: bool = False, mscale: float = 1.0, out_q=None,
         out_k=None, stream=None):
    """q [B, H, N, d] and k [B, H_kv, N, d] turned to their positions in one launch (fa_rope).

    k may be None: then only q's result is returned.  freq: a table of rope_frequencies() on the
    device; it rotates the first 2 * len(freq) elements of a row.  positions: int32 [B, N], or None
    for 0 .. N - 1.  Any strides with contiguous rows will do (slices of a joint projection);
    results are dense unless out_q, out_k are given, which may be q and k themselves.
    """
    return _rope(q, k, freq, positions, interleaved, mscale, out_q, out_k, 0, stream)


def rope_bwd(dq, dk, freq, positions=None, interleaved: bool = False, mscale: float = 1.0,
             out_q=None, out_k=None, stream=None):
    """The gradients of rope's q and k from those of its results (fa_rope with inverse set).

    out_q and out_k may be slices of the joint projection's gradient.
    """
    return _rope(dq, dk, freq, positions, interleaved, mscale, out_q, out_k, 1, stream)


def _paged_shapes(q, k_pages, v_pages, block_table, kv_len, q_start):
    """T, heads, d, num_pages, H_kv, page_size, B, max_pages, the dtype's code and the six page strides
    of a paged batch (q or k: [T, heads, d])."""
    shape, kshape, tshape, dt = q.shape, k_pages.shape, block_table.shape, q.dtype
    code = _DTYPES.get(dt)
    if code is None:
        _dtype_code(q)
    if len(shape) != 3:
        raise ValueError("tokens must be [T, heads, d]")
    T, H, d = shape
    if len(kshape) != 4 or kshape != v_pages.shape or kshape[3] != d \
            or k_pages.dtype is not dt or v_pages.dtype is not dt:
        raise ValueError("k_pages and v_pages must be [num_pages, H_kv, page_size, d] with the dtype "
                         "of the tokens")
    if len(tshape) != 2 or block_table.dtype is not _I32 or not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous int32 [B, max_pages]")
    B, max_pages = tshape
    _check_i32(kv_len, "kv_len", (B,))
    if q_start is not None:
        _check_i32(q_start, "q_start", (B + 1,))
    k0, k1, k2, ke = k_pages.stride()
    v0, v1, v2, ve = v_pages.stride()
    if ke != 1 or ve != 1:
        raise ValueError("the rows of the pages must be contiguous")
    num_pages, Hkv, page_size, _ = kshape
    return (T, H, d, num_pages, Hkv, page_size, B, max_pages, code, (k0, k1, k2, v0, v1, v2))


def paged_check(block_table, kv_len, q_start, num_pages: int, page_size: int,
                max_q: Optional[int] = None, tokens: Optional[int] = None) -> bool:
    """Whether CPU copies of a batch's index arrays are in range (fa_paged_check).

    tokens: T of the batch, when q_start is None (tokens / B each) or the batch is padded.
    """
    for name, t in (("block_table", block_table), ("kv_len", kv_len), ("q_start", q_start)):
        if t is not None and (t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous int32 CPU tensor")
    B, max_pages = block_table.shape
    if kv_len.shape != (B,) or (q_start is not None and q_start.shape != (B + 1,)):
        raise ValueError("kv_len must be [B] and q_start [B + 1]")
    if tokens is None:
        tokens = B if q_start is None else int(q_start[-1])
    rc = load().fa_paged_check(block_table.data_ptr(), kv_len.data_ptr(),
                               None if q_start is None else q_start.data_ptr(), tokens, B,
                               num_pages, page_size, max_pages, tokens if max_q is None else max_q)
    if rc == FA_ERR_INDEX:
        return False
    _check(rc, "fa_paged_check")
    return True


def paged_append(k, v, k_pages, v_pages, block_table, kv_len, q_start=None, q=None, out_q=None,
                 freq=None, positions=None, interleaved: bool = False, mscale: float = 1.0,
                 stream=None):
    """New tokens' k (rotated) and v [T, H_kv, d] into the paged cache (fa_paged_append).

    k_pages, v_pages: [num_pages, H_kv, page_size, d]; block_table int32 [B, max_pages]; kv_len int32
    [B], the new tokens included; q_start int32 [B + 1], or None for T / B tokens each.  With
    q [T, H, d] its rotated copy is returned (written to out_q, which may be q).  freq: a table of
    rope_frequencies(), or None for no rotation; positions int32 [T] rotates to other positions
    than the places in the cache.
    """
    dev = k.get_device()
    if dev < 0:
        raise ValueError("k must be a CUDA tensor")
    if stream is not None or dev != _current_device():
        return _elsewhere(lambda: paged_append(k, v, k_pages, v_pages, block_table, kv_len, q_start,
                                               q, out_q, freq, positions, interleaved, mscale),
                          stream, k.device, (k, v, k_pages, v_pages, block_table, kv_len, q_start, q,
                                             out_q, freq, positions))
    if v.get_device() != dev or k_pages.get_device() != dev or v_pages.get_device() != dev \
            or block_table.get_device() != dev or kv_len.get_device() != dev \
            or (q_start is not None and q_start.get_device() != dev) \
            or (q is not None and q.get_device() != dev) \
            or (freq is not None and freq.get_device() != dev) \
            or out_q is not None or positions is not None:
        _check_place(dev, v=v, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                     kv_len=kv_len, q_start=q_start, q=q, out_q=out_q, freq=freq,
                     positions=positions)
    T, Hkv, d, num_pages, pool_heads, page_size, B, max_pages, code, pages = \
        _paged_shapes(k, k_pages, v_pages, block_table, kv_len, q_start)
    dt = k.dtype
    if Hkv != pool_heads or v.shape != k.shape or v.dtype is not dt:
        raise ValueError("k and v must be [T, H_kv, d] with the H_kv and dtype of the pages")
    if positions is not None:
        _check_i32(positions, "positions", (T,))
    k0, k1, ke = k.stride()
    v0, v1, ve = v.stride()
    if q is not None:
        shape = q.shape
        if len(shape) != 3 or shape[0] != T or shape[2] != d or q.dtype is not dt:
            raise ValueError("q must be [T, H, d] with the dtype of k")
        H = shape[1]
        if out_q is None:
            out_q = _empty(shape, dtype=dt, device=q.device)
        elif out_q.shape != shape or out_q.dtype is not dt:
            raise ValueError("out_q must match q in shape and dtype")
        q0, q1, qe = q.stride()
        o0, o1, oe = out_q.stride()
        qp, op = q.data_ptr(), out_q.data_ptr()
    else:
        if out_q is not None:
            raise ValueError("out_q needs q")
        H, q0, q1, o0, o1, qp, op = Hkv, 0, 0, 8, 8, None, None
        qe = oe = 1
    if ke != 1 or ve != 1 or qe != 1 or oe != 1:
        raise ValueError("the rows of q, k and v must be contiguous")
    rc = load().fa_paged_append(
        qp, op, k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        _pack14(q0, q1, o0, o1, k0, k1, v0, v1, *pages), block_table.data_ptr(), kv_len.data_ptr(),
        None if q_start is None else q_start.data_ptr(),
        None if positions is None else positions.data_ptr(),
        None if freq is None else freq.data_ptr(), T, B, H, Hkv, d, num_pages, page_size, max_pages,
        0 if freq is None else _freq_table(freq), code, 1 if interleaved else 0, mscale, _raw(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_paged_append")
    return out_q


@functools.lru_cache(maxsize=1024)
def paged_workspace_bytes(T: int, B: int, H: int, H_kv: int, d: int, max_q: int, page_size: int,
                          max_pages: int) -> int:
    return int(load().fa_paged_attn_workspace_bytes(T, B, H, H_kv, d, max_q, page_size, max_pages))


def paged_attention(q, k_pages, v_pages, block_table, kv_len, q_start=None,
                    max_q: Optional[int] = None, scale: Optional[float] = None,
                    causal: bool = True, out=None, lse=None, workspace=None, stream=None):
    """O, LSE of every sequence's new tokens q [T, H, d] over its paged cache (fa_paged_attn).

    The cache (see paged_append) already holds the new tokens' keys and values; row i of the n new
    ones of sequence b sees keys j <= kv_len[b] - n + i, or with causal=False all kv_len[b].  max_q:
    the most new tokens that any sequence brings, when the caller knows it.  LSE is fp32 [T, H].
    """
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    if stream is not None or dev != _current_device():
        return _elsewhere(lambda: paged_attention(q, k_pages, v_pages, block_table, kv_len, q_start,
                                                  max_q, scale, causal, out, lse, workspace),
                          stream, q.device, (q, k_pages, v_pages, block_table, kv_len, q_start, out,
                                             lse, workspace))
    if k_pages.get_device() != dev or v_pages.get_device() != dev \
            or block_table.get_device() != dev or kv_len.get_device() != dev \
            or (q_start is not None and q_start.get_device() != dev) \
            or out is not None or lse is not None or workspace is not None:
        _check_place(dev, k_pages=k_pages, v_pages=v_pages, block_table=block_table, kv_len=kv_len,
                     q_start=q_start, out=out, lse=lse, workspace=workspace)
    T, H, d, num_pages, Hkv, page_size, B, max_pages, code, pages = \
        _paged_shapes(q, k_pages, v_pages, block_table, kv_len, q_start)
    if max_q is None:
        max_q = T if q_start is not None else max(T // max(B, 1), 1)
    device = q.device
    if out is None:
        out = _empty(q.shape, dtype=q.dtype, device=device)
    elif out.shape != q.shape or out.dtype is not q.dtype:
        raise ValueError("out must match q in shape and dtype")
    if lse is None:
        lse = _empty((T, H), dtype=_F32, device=device)
    elif lse.dtype is not _F32 or lse.shape != (T, H) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [T, H]")
    q0, q1, qe = q.stride()
    o0, o1, oe = out.stride()
    if qe != 1 or oe != 1:
        raise ValueError("the rows of q and out must be contiguous")
    nbytes = paged_workspace_bytes(T, B, H, Hkv, d, max_q, page_size, max_pages)
    if workspace is None:
        ws = None
        if nbytes > 0:
            workspace = _empty(nbytes, dtype=_U8, device=device)
            ws = workspace.data_ptr()
    elif not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace must be contiguous, of paged_workspace_bytes() bytes")
    else:
        ws = workspace.data_ptr()
    rc = load().fa_paged_attn(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), lse.data_ptr(),
        _pack10(q0, q1, o0, o1, *pages), block_table.data_ptr(), kv_len.data_ptr(),
        None if q_start is None else q_start.data_ptr(), T, B, H, Hkv, d, num_pages, page_size,
        max_pages, max_q, code, 1.0 / math.sqrt(d) if scale is None else scale, 1 if causal else 0,
        ws, nbytes, _raw(dev))
    if rc != FA_OK:
        raise FAError(rc, "fa_paged_attn")
    return out, lse


def sync_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load().fa_sync_status(_stream(stream)))


def debug_set_visit_log(buf: Optional[torch.Tensor]):
    if buf is None:
        _check(load().fa_debug_set_visit_log(None, 0), "fa_debug_set_visit_log")
    else:
        if buf.dtype != torch.uint8:
            raise TypeError("visit log must be uint8")
        _check(load().fa_debug_set_visit_log(_dev(buf, "visit_log"), buf.numel()),
               "fa_debug_set_visit_log")


def debug_set_wait_limit_ns(ns: int):
    _check(load().fa_debug_set_wait_limit_ns(int(ns)), "fa_debug_set_wait_limit_ns")


def debug_set_fault(mode: int):
    _check(load().fa_debug_set_fault(int(mode)), "fa_debug_set_fault")


def debug_set_dkdv_splits(splits: int):
    _check(load().fa_debug_set_dkdv_splits(int(splits)), "fa_debug_set_dkdv_splits")

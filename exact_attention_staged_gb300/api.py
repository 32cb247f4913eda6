"""Python binding of libfa.so: argument marshalling only (ctypes; the short calls of rotary positions,
the paged cache and beam selection through the extension csrc/binding.c, whose checks cost less time).

Every step of the attention path runs in the library's CUDA kernels; PyTorch supplies device
memory and the current stream.  There is no fallback: when libfa.so is missing or the device
is not an sm_103 GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import sysconfig
import threading
from typing import Optional, Tuple

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfa.so")
# with the suffix of this interpreter's extensions: one built for another Python is not loaded
BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                            "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

FA_FP16, FA_BF16, FA_FP32 = 0, 1, 2  # FA_FP32: beam_select's logits only
FA_OK, FA_ERR_INVALID, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = 0, -1, -2, -3, -4
FA_ERR_INTERNAL, FA_ERR_INDEX, FA_ERR_FULL = -5, -6, -7
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
    "fa_paged_reserve_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fa_paged_reserve": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp]),
    "fa_paged_fork": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "fa_paged_free": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "fa_paged_compact": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp]),
    "fa_paged_copy": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]),
    "fa_beam_select_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fa_beam_select": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _sz,
                            _vp]),
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
_binding = None


def _calls():
    """The extension that checks and makes the short calls (csrc/binding.c), set up once."""
    global _binding
    if _binding is None:
        lib = load()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing: build it with "
                               "`python -m exact_attention_staged_gb300.build`")
        from . import _binding as ext
        names = ("fa_rope", "fa_paged_append", "fa_paged_attn", "fa_paged_attn_workspace_bytes",
                 "fa_paged_reserve", "fa_paged_reserve_workspace_bytes", "fa_paged_fork", "fa_paged_free",
                 "fa_paged_compact", "fa_paged_copy", "fa_beam_select", "fa_beam_select_workspace_bytes")
        ext.setup(tuple(ctypes.cast(getattr(lib, n), _vp).value for n in names), torch.empty, _raw,
                  _current_device, torch.bfloat16, torch.float16, torch.int32, torch.int64, torch.float32,
                  torch.uint8, FAError)
        _binding = ext
    return _binding


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
    return torch.cuda.current_stream(dev).cuda_stream


if _raw_stream is not None:
    _raw = _raw_stream  # noqa: F811 (the same, without building a Stream object)


def _away(t, stream) -> bool:
    """Whether a call on tensor t has to leave the current device or stream."""
    if stream is not None:
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")
        return True
    return t.is_cuda and t.get_device() != _current_device()


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


def rope(q, k, freq, positions=None, interleaved: bool = False, mscale: float = 1.0, out_q=None,
         out_k=None, stream=None):
    """q [B, H, N, d] and k [B, H_kv, N, d] turned to their positions in one launch (fa_rope).

    k may be None: then only q's result is returned.  freq: a table of rope_frequencies() on the
    device; it rotates the first 2 * len(freq) elements of a row.  positions: int32 [B, N], or None
    for 0 .. N - 1.  Any strides with contiguous rows will do (slices of a joint projection);
    results are dense unless out_q, out_k are given, which may be q and k themselves.
    """
    if _away(q, stream):
        return _elsewhere(lambda: rope(q, k, freq, positions, interleaved, mscale, out_q, out_k),
                          stream, q.device, (q, k, freq, positions, out_q, out_k))
    return _calls().rope(q, k, freq, positions, interleaved, mscale, out_q, out_k, False)


def rope_bwd(dq, dk, freq, positions=None, interleaved: bool = False, mscale: float = 1.0,
             out_q=None, out_k=None, stream=None):
    """The gradients of rope's q and k from those of its results (fa_rope with inverse set).

    out_q and out_k may be slices of the joint projection's gradient.
    """
    if _away(dq, stream):
        return _elsewhere(lambda: rope_bwd(dq, dk, freq, positions, interleaved, mscale, out_q,
                                           out_k),
                          stream, dq.device, (dq, dk, freq, positions, out_q, out_k))
    return _calls().rope(dq, dk, freq, positions, interleaved, mscale, out_q, out_k, True)


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
        # at least one, as in a call: offsets that end below it are what is looked for
        tokens = B if q_start is None else max(int(q_start[-1]), 1)
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
    if _away(k, stream):
        return _elsewhere(lambda: paged_append(k, v, k_pages, v_pages, block_table, kv_len, q_start,
                                               q, out_q, freq, positions, interleaved, mscale),
                          stream, k.device, (k, v, k_pages, v_pages, block_table, kv_len, q_start, q,
                                             out_q, freq, positions))
    return _calls().paged_append(k, v, k_pages, v_pages, block_table, kv_len, q_start, q, out_q, freq,
                                 positions, interleaved, mscale)


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
    if _away(q, stream):
        return _elsewhere(lambda: paged_attention(q, k_pages, v_pages, block_table, kv_len, q_start,
                                                  max_q, scale, causal, out, lse, workspace),
                          stream, q.device, (q, k_pages, v_pages, block_table, kv_len, q_start, out,
                                             lse, workspace))
    return _calls().paged_attention(q, k_pages, v_pages, block_table, kv_len, q_start, max_q, scale,
                                    causal, out, lse, workspace)


def paged_reserve(block_table, kv_len, refs, page_size: int, q_start=None, tokens: Optional[int] = None,
                  copies=None, workspace=None, stream=None):
    """Pages of their own for a batch's new tokens (fa_paged_reserve).

    block_table int32 [B, max_pages] (-1: no page) and refs int32 [num_pages] (holders of each page) are
    updated.  kv_len and q_start as in paged_append; tokens: the batch's tokens (needed with q_start;
    None: one for each sequence).  Returns copies, int32 [3, B]: paged_copy's src, dst and rows for the
    pages that were shared and are partly filled.
    """
    if stream is None:
        done = _calls().paged_reserve(block_table, kv_len, refs, page_size, q_start, tokens, copies, workspace)
        if done is not NotImplemented:
            return done
    return _elsewhere(lambda: paged_reserve(block_table, kv_len, refs, page_size, q_start, tokens,
                                            copies, workspace),
                      stream, block_table.device, (block_table, kv_len, refs, q_start, copies,
                                                   workspace))


def paged_reserve_workspace_bytes(tokens: int, B: int, num_pages: int, page_size: int) -> int:
    return int(load().fa_paged_reserve_workspace_bytes(tokens, B, num_pages, page_size))


def paged_fork(block_table, parents, refs, kv_len=None, stream=None):
    """Row b of block_table (and kv_len) becomes what row parents[b] was; -1: empty (fa_paged_fork).

    parents: int32 [B], or [requests, beams] of B in all, as beam_select returns them.  refs follows.
    """
    if stream is None:
        done = _calls().paged_fork(block_table, parents, refs, kv_len)
        if done is not NotImplemented:
            return done
    return _elsewhere(lambda: paged_fork(block_table, parents, refs, kv_len), stream,
                      block_table.device, (block_table, parents, refs, kv_len))


def paged_free(block_table, keep_len, refs, page_size: int, stream=None):
    """Sequence b keeps the pages of its first keep_len[b] positions (int32 [B]; fa_paged_free)."""
    if stream is None:
        done = _calls().paged_free(block_table, keep_len, refs, page_size)
        if done is not NotImplemented:
            return done
    return _elsewhere(lambda: paged_free(block_table, keep_len, refs, page_size), stream,
                      block_table.device, (block_table, keep_len, refs))


def paged_compact(block_table, refs, moves=None, count=None, stream=None):
    """Moves the live pages to the front of the pool (fa_paged_compact).

    Returns moves, int32 [2, num_pages // 2 or more], and count, int32 [1]: paged_copy's src, dst and
    count, which move the data.  block_table and refs are updated.
    """
    if stream is None:
        done = _calls().paged_compact(block_table, refs, moves, count)
        if done is not NotImplemented:
            return done
    return _elsewhere(lambda: paged_compact(block_table, refs, moves, count), stream,
                      block_table.device, (block_table, refs, moves, count))


def paged_copy(k_pages, v_pages, src, dst, rows=None, count=None, stream=None):
    """The first rows[i] rows (None: all) of page src[i] to page dst[i], int32 [n] (fa_paged_copy).

    k_pages, v_pages: one layer's [num_pages, H_kv, page_size, d], or all layers' [L, num_pages, H_kv,
    page_size, d].  Pairs with a negative page are left out, and those from count (int32 [1]) on.
    """
    if stream is None:
        done = _calls().paged_copy(k_pages, v_pages, src, dst, rows, count)
        if done is not NotImplemented:
            return done
    return _elsewhere(lambda: paged_copy(k_pages, v_pages, src, dst, rows, count), stream,
                      k_pages.device, (k_pages, v_pages, src, dst, rows, count))


def beam_select(logits, scores, k: Optional[int] = None, finished=None, end_token: Optional[int] = None,
                out_scores=None, out_parents=None, out_tokens=None, out_finished=None, workspace=None,
                stream=None):
    """The k best continuations (None: as many as beams) of each request's beams (fa_beam_select).

    logits [B, W, V] of bf16, fp16 or fp32, any strides with contiguous rows; scores fp32 [B, W].
    finished: uint8 [B, W], beams that have ended: they offer end_token at their own score.  Returns
    scores (fp32), parents (int32, b * W + beam; -1: no candidate was left), tokens (int32) and finished
    (uint8), each [B, k], best first.
    """
    if stream is None:
        done = _calls().beam_select(logits, scores, k, finished, end_token, out_scores, out_parents,
                                    out_tokens, out_finished, workspace)
        if done is not NotImplemented:
            return done
    return _elsewhere(lambda: beam_select(logits, scores, k, finished, end_token, out_scores,
                                          out_parents, out_tokens, out_finished, workspace),
                      stream, logits.device, (logits, scores, finished, out_scores, out_parents,
                                              out_tokens, out_finished, workspace))


def beam_select_workspace_bytes(B: int, W: int, V: int, k: int) -> int:
    return int(load().fa_beam_select_workspace_bytes(B, W, V, k))


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

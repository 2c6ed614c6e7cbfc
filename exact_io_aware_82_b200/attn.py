"""Thin ctypes binding of libattn.so (the C ABI in include/attn.h).

Argument marshalling only: torch tensors are checked for device, dtype and contiguity and
passed as raw device pointers together with the current CUDA stream; every step of the
computation runs in the library's kernels.  Output and workspace tensors the caller does not
supply are allocated with torch (device memory is PyTorch's job here).  A non-zero status from
the library raises ``AttnError`` with the library's own message.  There is no fallback: if the
library is missing or no sm_100 device is present, calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

MASK_FULL, MASK_CAUSAL, MASK_SLIDING, MASK_LOCAL_GLOBAL = 0, 1, 2, 3
ATTN_OK = 0
ATTN_ERR_INVALID_ARG = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_CUDA = -3
ATTN_ERR_WORKSPACE = -4
ATTN_ERR_DEVICE_TIMEOUT = -5

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn.so")

# every symbol include/attn.h declares
EXPORTS = ("attn_abi_version", "attn_status_string", "attn_last_error_detail", "attn_fwd", "attn_fwd_f32",
           "attn_decode_workspace_bytes", "attn_decode", "attn_decode_num_splits",
           "attn_get_device_error", "attn_debug_timeout_probe", "attn_decode_noalloc",
           "attn_fwd_varlen", "attn_decode_paged", "attn_bwd", "attn_bwd_workspace_bytes", "attn_fwd_fp8",
           "attn_fwd_block_sparse", "attn_qk_norm_rope", "attn_qk_norm_rope_bwd",
           "attn_qk_norm_rope_bwd_workspace_bytes", "attn_qk_norm_rope_paged", "attn_page_update",
           "attn_decode_shared_prefix", "attn_decode_shared_prefix_workspace_bytes")

# size of the library-owned scratch array behind attn_decode_noalloc (include/attn.h)
DECODE_NOALLOC_MAX_BYTES = 64 << 20

_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = "%s: %s (status %d)" % (where, status_string(status), status)
        if status == ATTN_ERR_CUDA:
            msg += ": " + lib().attn_last_error_detail().decode()
        super().__init__(msg)


def lib():
    """Load libattn.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libattn.so is missing (%s): build it with "
                               "`python -m exact_io_aware_82_b200.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        L.attn_abi_version.argtypes, L.attn_abi_version.restype = [], i
        L.attn_status_string.argtypes, L.attn_status_string.restype = [i], ctypes.c_char_p
        L.attn_last_error_detail.argtypes, L.attn_last_error_detail.restype = [], ctypes.c_char_p
        L.attn_fwd.argtypes = [vp] * 5 + [i] * 9 + [f, vp]
        L.attn_fwd.restype = i
        L.attn_fwd_f32.argtypes = [vp] * 5 + [i] * 9 + [f, vp]
        L.attn_fwd_f32.restype = i
        L.attn_decode_workspace_bytes.argtypes = [i] * 6
        L.attn_decode_workspace_bytes.restype = ctypes.c_size_t
        L.attn_decode.argtypes = [vp] * 5 + [i] * 5 + [f, i, vp, ctypes.c_size_t, vp]
        L.attn_decode.restype = i
        L.attn_decode_num_splits.argtypes, L.attn_decode_num_splits.restype = [i] * 5, i
        L.attn_get_device_error.argtypes, L.attn_get_device_error.restype = [vp], i
        L.attn_debug_timeout_probe.argtypes = [ctypes.c_longlong, vp]
        L.attn_debug_timeout_probe.restype = i
        L.attn_decode_noalloc.argtypes = [vp] * 5 + [i] * 5 + [f, i, vp]
        L.attn_decode_noalloc.restype = i
        L.attn_fwd_varlen.argtypes = [vp] * 7 + [i] * 10 + [f, vp]
        L.attn_fwd_varlen.restype = i
        L.attn_decode_paged.argtypes = [vp] * 7 + [i] * 8 + [f, i, vp, ctypes.c_size_t, vp]
        L.attn_decode_paged.restype = i
        L.attn_fwd_fp8.argtypes = [vp] * 8 + [i] * 9 + [f, vp]
        L.attn_fwd_fp8.restype = i
        L.attn_fwd_block_sparse.argtypes = [vp] * 6 + [i] * 10 + [f, vp]
        L.attn_fwd_block_sparse.restype = i
        L.attn_bwd_workspace_bytes.argtypes = [i] * 7
        L.attn_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.attn_bwd.argtypes = [vp] * 9 + [i] * 9 + [f, vp, ctypes.c_size_t, vp]
        L.attn_bwd.restype = i
        L.attn_qk_norm_rope.argtypes = [vp] * 10 + [i] * 10 + [f, vp]
        L.attn_qk_norm_rope.restype = i
        L.attn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i]
        L.attn_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
        L.attn_qk_norm_rope_bwd.argtypes = [vp] * 14 + [i] * 10 + [f, vp, ctypes.c_size_t, vp]
        L.attn_qk_norm_rope_bwd.restype = i
        L.attn_qk_norm_rope_paged.argtypes = [vp] * 13 + [i] * 10 + [f, vp]
        L.attn_qk_norm_rope_paged.restype = i
        L.attn_page_update.argtypes = [vp] * 10 + [i] * 5 + [vp]
        L.attn_page_update.restype = i
        L.attn_decode_shared_prefix_workspace_bytes.argtypes = [i] * 7
        L.attn_decode_shared_prefix_workspace_bytes.restype = ctypes.c_size_t
        L.attn_decode_shared_prefix.argtypes = [vp] * 10 + [i] * 11 + [f, vp, ctypes.c_size_t, vp]
        L.attn_decode_shared_prefix.restype = i
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def abi_version() -> int:
    return int(lib().attn_abi_version())


def _stream_ptr(stream=None):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _check(t, name, dtype, ndim, shape=None):
    """Type, dtype, rank, contiguity and (if given) exact shape of one tensor argument."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %d-d tensor" % (name, ndim))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _check_out(t, name, dtype, shape):
    """An optional output / gradient tensor: None, or exactly the tensor the library writes."""
    if t is not None:
        _check(t, name, dtype, len(shape), shape)


def _check_workspace(ws, nbytes):
    import torch

    if ws is None:
        return
    _check(ws, "workspace", torch.uint8, 1)
    if ws.numel() < nbytes:
        raise ValueError("workspace holds %d bytes, the call needs %d" % (ws.numel(), nbytes))


def _device(stream, **tensors):
    """The one CUDA device that every given tensor (and the stream, if any) lives on.

    The library launches on the calling thread's current device with raw pointers, so a tensor
    on another device must be refused here rather than handed to a kernel."""
    devs = {t.device for t in tensors.values() if t is not None}
    if len(devs) != 1:
        raise ValueError("all tensors must be on one device, got %s" % ", ".join(
            "%s on %s" % (n, t.device) for n, t in tensors.items() if t is not None))
    dev = devs.pop()
    if dev.type != "cuda":
        raise ValueError("tensors must be CUDA tensors, got %s" % dev)
    if stream is not None and stream.device != dev:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, dev))
    return dev


def _raise(rc, where):
    if rc != ATTN_OK:
        raise AttnError(rc, where)


def attn_fwd(q, k, v, o=None, lse=None, mask_kind=MASK_FULL, window=0, n_sink=0, scale=None,
             return_lse=True, stream=None):
    """Exact attention forward on bf16 tensors q [B,Hq,Nq,d], k/v [B,Hkv,Nk,d].

    Returns (o, lse) with o bf16 [B,Hq,Nq,d] and lse fp32 [B,Hq,Nq] (None if not requested).
    """
    import torch

    _check(q, "q", torch.bfloat16, 4)
    B, Hq, Nq, d = q.shape
    _check(k, "k", torch.bfloat16, 4)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check_out(o, "o", torch.bfloat16, (B, Hq, Nq, d))
    _check_out(lse, "lse", torch.float32, (B, Hq, Nq))
    dev = _device(stream, q=q, k=k, v=v, o=o, lse=lse)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq, Nk, d,
                            int(mask_kind), int(window), int(n_sink), scale, _stream_ptr(stream))
    _raise(rc, "attn_fwd")
    return o, lse


def attn_fwd_block_sparse(q, k, v, block_mask, o=None, lse=None, mask_kind=MASK_FULL, window=0,
                          n_sink=0, scale=None, return_lse=True, stream=None):
    """attn_fwd under a fixed block-sparse layout: block_mask uint8 (or bool) [1 or Hq,
    ceil(Nq/128), ceil(Nk/128)] selects the 128 x 128 blocks each head attends (one layout for
    every head when its first dimension is 1).  Returns (o, lse) as attn_fwd."""
    import torch

    _check(q, "q", torch.bfloat16, 4)
    B, Hq, Nq, d = q.shape
    _check(k, "k", torch.bfloat16, 4)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.bfloat16, 4, (B, Hkv, Nk, d))
    if isinstance(block_mask, torch.Tensor) and block_mask.dtype == torch.bool:
        block_mask = block_mask.view(torch.uint8)
    _check(block_mask, "block_mask", torch.uint8, 3)
    shape = (block_mask.shape[0], -(-Nq // 128), -(-Nk // 128))
    if block_mask.shape[0] not in (1, Hq):
        raise ValueError("block_mask must have 1 or Hq = %d layouts, got %d" % (Hq, block_mask.shape[0]))
    _check(block_mask, "block_mask", torch.uint8, 3, shape)
    _check_out(o, "o", torch.bfloat16, (B, Hq, Nq, d))
    _check_out(lse, "lse", torch.float32, (B, Hq, Nq))
    dev = _device(stream, q=q, k=k, v=v, block_mask=block_mask, o=o, lse=lse)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_fwd_block_sparse(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                         _ptr(block_mask), int(block_mask.shape[0]), B, Hq, Hkv,
                                         Nq, Nk, d, int(mask_kind), int(window), int(n_sink),
                                         scale, _stream_ptr(stream))
    _raise(rc, "attn_fwd_block_sparse")
    return o, lse


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, o=None, lse=None,
                    mask_kind=MASK_FULL, window=0, n_sink=0, scale=None, return_lse=True,
                    stream=None):
    """Packed variable-length forward: q [total_q, Hq, d], k/v [total_k, Hkv, d] bf16;
    cu_seqlens_q / cu_seqlens_k int32 CUDA tensors of num_seqs + 1 offsets.

    Returns (o [total_q, Hq, d] bf16, lse [total_q, Hq] fp32).  Rows outside every sequence are
    left as they were in ``o`` / ``lse`` (allocated uninitialised when not given).
    """
    import torch

    _check(q, "q", torch.bfloat16, 3)
    total_q, Hq, d = q.shape
    _check(k, "k", torch.bfloat16, 3)
    total_k, Hkv = k.shape[0], k.shape[1]
    _check(k, "k", torch.bfloat16, 3, (total_k, Hkv, d))
    _check(v, "v", torch.bfloat16, 3, (total_k, Hkv, d))
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    num_seqs = cu_seqlens_q.numel() - 1
    if num_seqs < 0:
        raise ValueError("cu_seqlens_q needs num_seqs + 1 >= 1 offsets")
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1, (num_seqs + 1,))
    _check_out(o, "o", torch.bfloat16, (total_q, Hq, d))
    _check_out(lse, "lse", torch.float32, (total_q, Hq))
    dev = _device(stream, q=q, k=k, v=v, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
                  o=o, lse=lse)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((total_q, Hq), dtype=torch.float32, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                   _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), num_seqs, Hq, Hkv,
                                   total_q, total_k, int(max_seqlen_q), d, int(mask_kind),
                                   int(window), int(n_sink), scale, _stream_ptr(stream))
    _raise(rc, "attn_fwd_varlen")
    return o, lse


def attn_fwd_fp8(q, k, v, descale_q, descale_k, descale_v, o=None, lse=None,
                 mask_kind=MASK_FULL, window=0, n_sink=0, scale=None, return_lse=True,
                 stream=None):
    """E4M3 forward: q [B,Hq,Nq,d], k, v [B,Hkv,Nk,d] as uint8 (or float8_e4m3fn) codes;
    descale_q [B,Hq], descale_k / descale_v [B,Hkv] fp32 CUDA tensors.  Returns (o bf16, lse)."""
    import torch

    def codes(t, n):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % n)
        if t.dtype == getattr(torch, "float8_e4m3fn", None):
            t = t.view(torch.uint8)
        _check(t, n, torch.uint8, 4)
        return t

    q, k, v = codes(q, "q"), codes(k, "k"), codes(v, "v")
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.uint8, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.uint8, 4, (B, Hkv, Nk, d))
    _check(descale_q, "descale_q", torch.float32, 2, (B, Hq))
    _check(descale_k, "descale_k", torch.float32, 2, (B, Hkv))
    _check(descale_v, "descale_v", torch.float32, 2, (B, Hkv))
    _check_out(o, "o", torch.bfloat16, (B, Hq, Nq, d))
    _check_out(lse, "lse", torch.float32, (B, Hq, Nq))
    dev = _device(stream, q=q, k=k, v=v, descale_q=descale_q, descale_k=descale_k,
                  descale_v=descale_v, o=o, lse=lse)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty((B, Hq, Nq, d), dtype=torch.bfloat16, device=dev)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(descale_q),
                                _ptr(descale_k), _ptr(descale_v), B, Hq, Hkv, Nq, Nk, d,
                                int(mask_kind), int(window), int(n_sink), scale,
                                _stream_ptr(stream))
    _raise(rc, "attn_fwd_fp8")
    return o, lse


def attn_fwd_f32(q, k, v, o=None, lse=None, mask_kind=MASK_FULL, window=0, n_sink=0, scale=None,
                 return_lse=True, stream=None):
    """Exact attention forward on fp32 tensors (same shapes and rules as attn_fwd)."""
    import torch

    _check(q, "q", torch.float32, 4)
    B, Hq, Nq, d = q.shape
    _check(k, "k", torch.float32, 4)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.float32, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.float32, 4, (B, Hkv, Nk, d))
    _check_out(o, "o", torch.float32, (B, Hq, Nq, d))
    _check_out(lse, "lse", torch.float32, (B, Hq, Nq))
    dev = _device(stream, q=q, k=k, v=v, o=o, lse=lse)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nq,
                                Nk, d, int(mask_kind), int(window), int(n_sink), scale,
                                _stream_ptr(stream))
    _raise(rc, "attn_fwd_f32")
    return o, lse


def attn_bwd_workspace_bytes(B, Hq, Nq, Nk, mask_kind=MASK_FULL, window=0, n_sink=0) -> int:
    return int(lib().attn_bwd_workspace_bytes(B, Hq, Nq, Nk, int(mask_kind), int(window),
                                              int(n_sink)))


def attn_bwd(q, k, v, o, lse, dout, mask_kind=MASK_FULL, window=0, n_sink=0, scale=None,
             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of attn_fwd: returns (dq, dk, dv), bf16 with the shapes of q, k, v.

    o and lse are the forward's outputs for the same q, k, v, mask and scale; dout = dL/dO.
    """
    import torch

    _check(q, "q", torch.bfloat16, 4)
    B, Hq, Nq, d = q.shape
    _check(k, "k", torch.bfloat16, 4)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check(o, "o", torch.bfloat16, 4, (B, Hq, Nq, d))
    _check(dout, "dout", torch.bfloat16, 4, (B, Hq, Nq, d))
    _check(lse, "lse", torch.float32, 3, (B, Hq, Nq))
    _check_out(dq, "dq", torch.bfloat16, (B, Hq, Nq, d))
    _check_out(dk, "dk", torch.bfloat16, (B, Hkv, Nk, d))
    _check_out(dv, "dv", torch.bfloat16, (B, Hkv, Nk, d))
    _check_workspace(workspace, 0)
    dev = _device(stream, q=q, k=k, v=v, o=o, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv,
                  workspace=workspace)
    with torch.cuda.device(dev):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        if workspace is None:
            workspace = torch.empty(max(attn_bwd_workspace_bytes(B, Hq, Nq, Nk, mask_kind, window,
                                                                 n_sink), 16),
                                    dtype=torch.uint8, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
                            _ptr(dk), _ptr(dv), B, Hq, Hkv, Nq, Nk, d, int(mask_kind),
                            int(window), int(n_sink), scale, _ptr(workspace), workspace.numel(),
                            _stream_ptr(stream))
    _raise(rc, "attn_bwd")
    return dq, dk, dv


def attn_decode_workspace_bytes(B, Hq, Hkv, Nk, d, num_splits=0) -> int:
    return int(lib().attn_decode_workspace_bytes(B, Hq, Hkv, Nk, d, num_splits))


def attn_decode_num_splits(B, Hq, Hkv, Nk, d) -> int:
    return int(lib().attn_decode_num_splits(B, Hq, Hkv, Nk, d))


def _decode_query(q):
    import torch

    _check(q, "q", torch.bfloat16, 4)
    B, Hq, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes one query token per sequence (q.shape[2] == 1)")
    return B, Hq, d


def attn_decode(q, k, v, o=None, lse=None, scale=None, num_splits=0, workspace=None,
                return_lse=True, stream=None):
    """Split-K decode: q [B,Hq,1,d] bf16 against the cache k/v [B,Hkv,Nk,d] bf16.

    Returns (o [B,Hq,1,d] bf16, lse [B,Hq] fp32).  ``workspace`` (a uint8 CUDA tensor of at
    least attn_decode_workspace_bytes(...) bytes) is allocated with torch when not given.
    """
    import torch

    B, Hq, d = _decode_query(q)
    _check(k, "k", torch.bfloat16, 4)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check_out(o, "o", torch.bfloat16, (B, Hq, 1, d))
    _check_out(lse, "lse", torch.float32, (B, Hq))
    _check_workspace(workspace, 0)
    dev = _device(stream, q=q, k=k, v=v, o=o, lse=lse, workspace=workspace)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        if workspace is None:
            nbytes = attn_decode_workspace_bytes(B, Hq, Hkv, Nk, d, num_splits)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Nk, d,
                               scale, int(num_splits), _ptr(workspace), workspace.numel(),
                               _stream_ptr(stream))
    _raise(rc, "attn_decode")
    return o, lse


def attn_decode_paged(q, k_cache, v_cache, block_table, seq_lens, max_seq_len, o=None, lse=None,
                      scale=None, num_splits=0, workspace=None, return_lse=True, stream=None):
    """Decode against a paged cache.

    q [B,Hq,1,d] bf16; k_cache/v_cache [num_pages,page_size,Hkv,d] bf16; block_table
    [B,max_pages_per_seq] int32; seq_lens [B] int32 (device); max_seq_len an int >= every length.
    Returns (o [B,Hq,1,d] bf16, lse [B,Hq] fp32).
    """
    import torch

    B, Hq, d = _decode_query(q)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    num_pages, page_size, Hkv, dk = k_cache.shape
    if dk != d:
        raise ValueError("k_cache and v_cache must both be [num_pages, page_size, Hkv, d]")
    _check(v_cache, "v_cache", torch.bfloat16, 4, k_cache.shape)
    _check(block_table, "block_table", torch.int32, 2)
    if block_table.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    _check(seq_lens, "seq_lens", torch.int32, 1, (B,))
    _check_out(o, "o", torch.bfloat16, (B, Hq, 1, d))
    _check_out(lse, "lse", torch.float32, (B, Hq))
    _check_workspace(workspace, 0)
    dev = _device(stream, q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table,
                  seq_lens=seq_lens, o=o, lse=lse, workspace=workspace)
    max_seq_len = int(max_seq_len)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        if workspace is None:
            nbytes = attn_decode_workspace_bytes(B, Hq, Hkv, max_seq_len, d, num_splits)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                                     _ptr(block_table), _ptr(seq_lens), B, Hq, Hkv, num_pages,
                                     page_size, block_table.shape[1], max_seq_len, d, scale,
                                     int(num_splits), _ptr(workspace), workspace.numel(),
                                     _stream_ptr(stream))
    _raise(rc, "attn_decode_paged")
    return o, lse


def attn_decode_noalloc(q, k, v, o=None, lse=None, scale=None, num_splits=0, return_lse=True,
                        stream=None):
    """attn_decode without a workspace, for callers that cannot allocate device memory: the
    split partials live in a fixed library-owned device array of DECODE_NOALLOC_MAX_BYTES
    (shared by every call on the device, so calls that overlap on the GPU race).  Raises
    AttnError(ATTN_ERR_WORKSPACE) when the call would need more than that array."""
    import torch

    B, Hq, d = _decode_query(q)
    _check(k, "k", torch.bfloat16, 4)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check(k, "k", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check(v, "v", torch.bfloat16, 4, (B, Hkv, Nk, d))
    _check_out(o, "o", torch.bfloat16, (B, Hq, 1, d))
    _check_out(lse, "lse", torch.float32, (B, Hq))
    dev = _device(stream, q=q, k=k, v=v, o=o, lse=lse)
    with torch.cuda.device(dev):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and return_lse:
            lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
        scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
        rc = lib().attn_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv,
                                       Nk, d, scale, int(num_splits), _stream_ptr(stream))
    _raise(rc, "attn_decode_noalloc")
    return o, lse


# ---- around attention ------------------------------------------------------------------------
# A decode step makes several of these calls, so their checks spend little on arguments that are right.

def _expect(t, name, dtype, shape):
    """_check of one contiguous tensor of exactly this shape."""
    import torch

    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _check(t, name, dtype, len(shape), shape)


def _expect_out(t, name, dtype, shape):
    if t is not None:
        _expect(t, name, dtype, shape)


def _expect_view(t, name, dtype, shape, written=False):
    """A strided tensor argument: type, dtype, shape and a contiguous last dimension; one that is
    written must not hold an element twice (an expanded or self-overlapping view)."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    if written and not t.is_contiguous():
        end = 1
        for step, n in sorted((t.stride(i), t.shape[i]) for i in range(t.dim()) if t.shape[i] > 1):
            if step < end:
                raise ValueError("%s overlaps itself: a tensor that is written needs rows of its own" % name)
            end = step * (n - 1) + end


_MOST = 0x7fffffff  # of a size: the C ABI takes 32 bits, and ctypes would cut a larger one down without a word


def _refuse_sizes(**sizes):
    for n, v in sizes.items():
        if not -_MOST <= v <= _MOST:
            raise ValueError("%s must fit in 32 bits, got %d" % (n, v))


def _one_device(stream, **tensors):
    """The device of all tensors (and of the stream), as _device."""
    index = None
    for t in tensors.values():
        if t is not None:
            i = t.get_device()  # -1 where it is not a CUDA tensor
            if i != index:
                if index is not None or i < 0:
                    return _device(stream, **tensors)  # refuses them
                index, first = i, t
    return first.device if stream is None else _device(stream, **tensors)


def _new(dev, stream, dtype, *shape):
    """Memory for an output or a workspace of a call on `stream` (None: the current one), taken from
    that stream's pool: what the current stream freed last may still be in use there."""
    import torch

    if stream is None:  # (sizes one by one: a tuple takes a microsecond longer)
        return torch.empty(*shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=dev)
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _call(fn, where, dev, stream, *args):
    """fn(*args, stream) with dev current; raises on a status."""
    import torch

    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, _raw_stream(dev.index, stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev.index, stream))
    if rc != ATTN_OK:
        raise AttnError(rc, where)


def _raw_stream(index, stream):
    import torch

    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _at(t):
    return t.data_ptr() if t is not None else None


@functools.lru_cache(maxsize=1024)
def attn_decode_shared_prefix_workspace_bytes(B, Hq, Hkv, num_groups, max_prefix_len, max_seq_len,
                                              d) -> int:
    if max(B, Hq, Hkv, num_groups, max_prefix_len, max_seq_len, d) > _MOST:
        return 0  # as for every size that the call refuses
    return int(lib().attn_decode_shared_prefix_workspace_bytes(B, Hq, Hkv, num_groups, max_prefix_len,
                                                               max_seq_len, d))


def attn_decode_shared_prefix(q, k_cache, v_cache, prefix_table, prefix_lens, group_starts,
                              block_table, seq_lens, max_prefix_len, max_seq_len, o=None, lse=None,
                              scale=None, workspace=None, return_lse=True, stream=None):
    """Decode for sequences behind shared prefixes, over a paged cache.

    q [B,Hq,1,d] bf16; k_cache/v_cache [num_pages,page_size,Hkv,d] bf16; prefix g has prefix_lens[g]
    keys in pages prefix_table[g] ([num_groups,max_prefix_pages] int32) and is shared by sequences
    group_starts[g] .. group_starts[g+1]-1 (int32 [num_groups+1], device); block_table
    [B,max_pages_per_seq] and seq_lens [B] int32 hold each sequence's own keys.  max_prefix_len and
    max_seq_len are ints >= every length.  Returns (o [B,Hq,1,d] bf16, lse [B,Hq] fp32).
    Row b of q is sequence b's query (attn_qk_norm_rope_paged returns a row per new token: gather first).
    """
    import torch

    B, Hq, d = _decode_query(q)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    num_pages, page_size, Hkv, dk = k_cache.shape
    if dk != d:
        raise ValueError("k_cache and v_cache must both be [num_pages, page_size, Hkv, d]")
    _expect(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    _check(prefix_table, "prefix_table", torch.int32, 2)
    num_groups = prefix_table.shape[0]
    _expect(prefix_lens, "prefix_lens", torch.int32, (num_groups,))
    _expect(group_starts, "group_starts", torch.int32, (num_groups + 1,))
    _check(block_table, "block_table", torch.int32, 2)
    if block_table.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    _expect(seq_lens, "seq_lens", torch.int32, (B,))
    _expect_out(o, "o", torch.bfloat16, (B, Hq, 1, d))
    _expect_out(lse, "lse", torch.float32, (B, Hq))
    _check_workspace(workspace, 0)
    max_prefix_len, max_seq_len = int(max_prefix_len), int(max_seq_len)
    prefix_pages, seq_pages = prefix_table.shape[1], block_table.shape[1]
    if not (-_MOST <= max_prefix_len <= _MOST and -_MOST <= max_seq_len <= _MOST and prefix_pages <= _MOST
            and seq_pages <= _MOST):
        _refuse_sizes(max_prefix_len=max_prefix_len, max_seq_len=max_seq_len, max_prefix_pages=prefix_pages,
                      max_pages_per_seq=seq_pages)
    dev = _one_device(stream, q=q, k_cache=k_cache, v_cache=v_cache, prefix_table=prefix_table,
                      prefix_lens=prefix_lens, group_starts=group_starts, block_table=block_table,
                      seq_lens=seq_lens, o=o, lse=lse, workspace=workspace)
    if o is None:
        o = _new(dev, stream, torch.bfloat16, B, Hq, 1, d)
    if lse is None and return_lse:
        lse = _new(dev, stream, torch.float32, B, Hq)
    if workspace is None:
        nbytes = attn_decode_shared_prefix_workspace_bytes(B, Hq, Hkv, num_groups, max_prefix_len,
                                                           max_seq_len, d)
        workspace = _new(dev, stream, torch.uint8, max(nbytes, 16))
    _call(lib().attn_decode_shared_prefix, "attn_decode_shared_prefix", dev, stream, q.data_ptr(),
          k_cache.data_ptr(), v_cache.data_ptr(), o.data_ptr(), _at(lse), prefix_table.data_ptr(),
          prefix_lens.data_ptr(), group_starts.data_ptr(), block_table.data_ptr(),
          seq_lens.data_ptr(), B, Hq, Hkv, num_groups, num_pages, page_size, prefix_pages,
          max_prefix_len, seq_pages, max_seq_len, d,
          1.0 / math.sqrt(d) if scale is None else float(scale), workspace.data_ptr(),
          workspace.numel())
    return o, lse


def _bhn(t):
    """(b, h, n) element strides of a [B,H,N,d] or packed [T,H,d] tensor."""
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[1], s[0])


@functools.lru_cache(maxsize=64)
def _section_array(sections, pairs):
    if not 1 <= len(sections) <= 4 or min(sections) < 0 or sum(sections) != pairs:
        raise ValueError("sections must be 1 to 4 counts of pairs that add up to rope.shape[1] / 2 = %d, got %s"
                         % (pairs, list(sections)))
    return (ctypes.c_int * len(sections))(*sections)


class _QkShapes:
    """Shapes of a norm + rotation call, dense [B,H,N,d] or packed [T,H,d]: checks q, k, the weights,
    the table, the positions and the sections, and keeps what the library is told about them."""

    def __init__(self, q, k, q_weight, k_weight, rope, positions, sections):
        import torch

        if not isinstance(q, torch.Tensor) or not isinstance(k, torch.Tensor):
            raise TypeError("q and k must be torch.Tensors")
        dtype = q.dtype
        if dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise TypeError("q must be torch.bfloat16 or torch.float32, got %s" % dtype)
        q_shape, k_shape = q.shape, k.shape
        if len(q_shape) not in (3, 4) or len(k_shape) != len(q_shape):
            raise ValueError("q and k must both be [B, H, N, d] or both packed [tokens, H, d]")
        self.dtype, self.code = dtype, 0 if dtype is torch.bfloat16 else 1
        self.dense = len(q_shape) == 4
        if self.dense:
            B, Hq, N, d = q_shape
            Hkv = k_shape[1]
            k_want = (B, Hkv, N, d)
        else:
            B, (N, Hq, d) = 1, q_shape
            Hkv = k_shape[1]
            k_want = (N, Hkv, d)
        self.q_shape, self.k_shape = q_shape, k_want
        qs, ks = q.stride(), k.stride()
        if qs[-1] != 1 or k.dtype is not dtype or k_shape != k_want or ks[-1] != 1:
            _expect_view(q, "q", dtype, q_shape)
            _expect_view(k, "k", dtype, k_want)
        # (b, h, n) strides
        self.qk = qs[:3] + ks[:3] if self.dense else (0, qs[1], qs[0], 0, ks[1], ks[0])
        if q_weight is not None:
            _expect(q_weight, "q_weight", dtype, (d,))
        if k_weight is not None:
            _expect(k_weight, "k_weight", dtype, (d,))
        _check(rope, "rope", torch.float32, 2)
        max_pos, rot = rope.shape
        axes = 1
        self.sections = None
        lead = ()
        if sections is not None:
            self.sections = _section_array(tuple(map(int, sections)), rot // 2)
            axes = len(sections)
            lead = (axes,)
        if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32:
            raise TypeError("positions must be a torch.int32 tensor")
        shape = positions.shape
        per_row = self.dense and shape == lead + (B, N)
        if not per_row and shape != lead + (N,):
            raise ValueError("positions must have shape %s%s, got %s" % (
                lead + (N,), " or %s" % (lead + (B, N),) if self.dense else "", tuple(shape)))
        strides = positions.stride()
        if N > 1 and strides[-1] != 1:
            raise ValueError("positions must be contiguous in its last dimension")
        self.pos = (strides[0] if lead else 0, strides[-2] if per_row else 0)
        self.N, self.Hq, self.Hkv, self.d = N, Hq, Hkv, d
        # what the library is told: sizes, and from the head size on the rest
        self.sizes = (B, N, Hq, Hkv)
        self.rest = (d, rot, max_pos, axes)


# host arrays of long long: strides of the forward, backward and paged calls
_STRIDES, _STRIDES_BWD, _STRIDES_PAGED = (struct.Struct("%dq" % n).pack for n in (14, 20, 13))


def attn_qk_norm_rope(q, k, q_weight, k_weight, rope, positions, sections=None, interleaved=False,
                      eps=1e-6, q_out=None, k_out=None, stream=None):
    """Queries and keys normalised per head, weighted and rotated by position, in one pass.

    q [B,Hq,N,d], k [B,Hkv,N,d] (attn_fwd's layout) or packed q [T,Hq,d], k [T,Hkv,d]
    (attn_fwd_varlen's), bf16 or fp32, d 64 or 128; any strides with d contiguous and 16-byte rows, as
    views into a fused projection have.  q_weight, k_weight [d] in the same type, or None where that
    side is not normalised.  rope fp32 [max_pos, rot_dim]: cosines, then sines, of each position's
    angles; rot_dim a multiple of 16 up to d.  positions int32 [N] or [B,N] ([T] packed); with sections
    (the rotated pairs of each position axis) [axes,N] or [axes,B,N] ([axes,T]).  interleaved pairs
    columns (2i, 2i+1) instead of (i, i + rot_dim/2).

    Returns (q_out, k_out), contiguous unless given; an output may be its input (the same view), and must not
    overlap the inputs otherwise.
    """
    s = _QkShapes(q, k, q_weight, k_weight, rope, positions, sections)
    if q_out is not None:
        _expect_view(q_out, "q_out", s.dtype, s.q_shape, written=True)
    if k_out is not None:
        _expect_view(k_out, "k_out", s.dtype, s.k_shape, written=True)
    dev = _one_device(stream, q=q, k=k, q_weight=q_weight, k_weight=k_weight, rope=rope,
                      positions=positions, q_out=q_out, k_out=k_out)
    if q_out is None:
        q_out = _new(dev, stream, s.dtype, *s.q_shape)
    if k_out is None:
        k_out = _new(dev, stream, s.dtype, *s.k_shape)
    _call(lib().attn_qk_norm_rope, "attn_qk_norm_rope", dev, stream, q.data_ptr(), k.data_ptr(),
          q_out.data_ptr(), k_out.data_ptr(), _at(q_weight), _at(k_weight), rope.data_ptr(),
          positions.data_ptr(), _STRIDES(*s.qk, *_bhn(q_out), *_bhn(k_out), *s.pos), s.sections,
          s.code, *s.sizes, *s.rest, 1 if interleaved else 0, float(eps))
    return q_out, k_out


@functools.lru_cache(maxsize=16)
def attn_qk_norm_rope_bwd_workspace_bytes(d) -> int:
    return int(lib().attn_qk_norm_rope_bwd_workspace_bytes(d))


def attn_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, rope, positions, sections=None,
                          interleaved=False, eps=1e-6, dq=None, dk=None, dq_weight=None,
                          dk_weight=None, workspace=None, stream=None):
    """Gradient of attn_qk_norm_rope: dq_out, dk_out are the gradients of its outputs (attn_bwd's dq
    and dk), the other arguments those of the call.

    Returns (dq, dk, dq_weight, dk_weight): dq, dk like q, k (contiguous unless given), the weights'
    gradients fp32 [d], None where there is no weight.
    """
    import torch

    s = _QkShapes(q, k, q_weight, k_weight, rope, positions, sections)
    _expect_view(dq_out, "dq_out", s.dtype, s.q_shape)
    _expect_view(dk_out, "dk_out", s.dtype, s.k_shape)
    if dq is not None:
        _expect_view(dq, "dq", s.dtype, s.q_shape, written=True)
    if dk is not None:
        _expect_view(dk, "dk", s.dtype, s.k_shape, written=True)
    for t, w, n in ((dq_weight, q_weight, "dq_weight"), (dk_weight, k_weight, "dk_weight")):
        if t is not None:
            if w is None:
                raise ValueError("%s is given but the weight is not" % n)
            _expect(t, n, torch.float32, (s.d,))
    _check_workspace(workspace, 0)
    dev = _one_device(stream, q=q, k=k, dq_out=dq_out, dk_out=dk_out, q_weight=q_weight,
                      k_weight=k_weight, rope=rope, positions=positions, dq=dq, dk=dk,
                      dq_weight=dq_weight, dk_weight=dk_weight, workspace=workspace)
    if dq is None:
        dq = _new(dev, stream, s.dtype, *s.q_shape)
    if dk is None:
        dk = _new(dev, stream, s.dtype, *s.k_shape)
    if dq_weight is None and q_weight is not None:
        dq_weight = _new(dev, stream, torch.float32, s.d)
    if dk_weight is None and k_weight is not None:
        dk_weight = _new(dev, stream, torch.float32, s.d)
    if workspace is None:
        workspace = _new(dev, stream, torch.uint8, max(attn_qk_norm_rope_bwd_workspace_bytes(s.d), 16))
    _call(lib().attn_qk_norm_rope_bwd, "attn_qk_norm_rope_bwd", dev, stream, q.data_ptr(), k.data_ptr(),
          dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), _at(q_weight),
          _at(k_weight), _at(dq_weight), _at(dk_weight), rope.data_ptr(), positions.data_ptr(),
          _STRIDES_BWD(*s.qk, *_bhn(dq_out), *_bhn(dk_out), *_bhn(dq), *_bhn(dk), *s.pos),
          s.sections, s.code, *s.sizes, *s.rest, 1 if interleaved else 0, float(eps),
          workspace.data_ptr(), workspace.numel())
    return dq, dk, dq_weight, dk_weight


def attn_qk_norm_rope_paged(q, k, v, q_weight, k_weight, rope, positions, slots, k_cache, v_cache,
                            sections=None, interleaved=False, eps=1e-6, q_out=None, stream=None):
    """attn_qk_norm_rope for serving: q [T,Hq,d] goes to q_out, k (normalised, rotated) and v
    [T,Hkv,d] into rows slots[t] of the paged cache k_cache / v_cache [num_pages,page_size,Hkv,d]
    (bf16, d 128; q, k, v any strides with d contiguous and 16-byte rows).  slots int32 [T], distinct;
    a token with a negative slot is left out.  Returns q_out [T,Hq,d], contiguous unless given: as
    [T,Hq,1,d] (unsqueeze(2)) it is the decode calls' q.  Rows of left-out tokens keep what q_out held.
    """
    import torch

    s = _QkShapes(q, k, q_weight, k_weight, rope, positions, sections)
    if s.dense or s.code != 0:
        raise ValueError("q, k and v must be packed bf16 [tokens, H, d] tensors")
    _expect_view(v, "v", s.dtype, s.k_shape)
    _expect(slots, "slots", torch.int32, (s.N,))
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    num_pages, page_size = k_cache.shape[:2]
    _expect(k_cache, "k_cache", torch.bfloat16, (num_pages, page_size, s.Hkv, s.d))
    _expect(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    if q_out is not None:
        _expect_view(q_out, "q_out", s.dtype, s.q_shape, written=True)
    dev = _one_device(stream, q=q, k=k, v=v, q_weight=q_weight, k_weight=k_weight, rope=rope,
                      positions=positions, slots=slots, k_cache=k_cache, v_cache=v_cache, q_out=q_out)
    if q_out is None:
        q_out = _new(dev, stream, s.dtype, *s.q_shape)
    _call(lib().attn_qk_norm_rope_paged, "attn_qk_norm_rope_paged", dev, stream, q.data_ptr(), k.data_ptr(),
          v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _at(q_weight),
          _at(k_weight), rope.data_ptr(), positions.data_ptr(), slots.data_ptr(),
          _STRIDES_PAGED(*s.qk, *_bhn(v), *_bhn(q_out), s.pos[0]), s.sections, s.N, s.Hq, s.Hkv,
          num_pages, page_size, *s.rest, 1 if interleaved else 0, float(eps))
    return q_out


def attn_page_update(block_table, old_lens, new_lens, free_pages, ring, page_size, max_tokens,
                     pos_offset=None, ring_out=None, cu_seqlens=None, slots=None, positions=None,
                     stream=None):
    """One step of a paged cache's bookkeeping, on the device: requests grow from old_lens to
    new_lens (int32 [B]), shrink (rejected tokens, 0 for an ended request) or stay.

    block_table int32 [B,max_pages_per_seq] and free_pages int32 [num_pages] (a ring of free page
    numbers) are updated in place; ring int64 [3] holds the ring's head and tail (free entries are
    head .. tail-1 modulo num_pages; a fresh pool is arange(num_pages) with [0, num_pages, 0]).

    Returns (ring_out int64 [3], cu_seqlens int32 [B+1], slots int32 [max_tokens], positions int32
    [max_tokens]): ring for the next step, with the number of pages missing in ring_out[2] (0: done;
    > 0: the pool is short, -1: invalid lengths; nothing was changed then), the new tokens' offsets
    per request, and each new token's cache row and position (plus pos_offset[b], int32 [B]); -1 and
    0 behind the last.  ring_out must not be ring.
    """
    import torch

    _check(block_table, "block_table", torch.int32, 2)
    B, max_pages = block_table.shape
    _expect(old_lens, "old_lens", torch.int32, (B,))
    _expect(new_lens, "new_lens", torch.int32, (B,))
    _check(free_pages, "free_pages", torch.int32, 1)
    _expect(ring, "ring", torch.int64, (3,))
    max_tokens, page_size = int(max_tokens), int(page_size)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    num_pages = free_pages.shape[0]
    if not (max_tokens <= _MOST and -_MOST <= page_size <= _MOST and max_pages <= _MOST and num_pages <= _MOST):
        _refuse_sizes(max_tokens=max_tokens, page_size=page_size, max_pages_per_seq=max_pages, num_pages=num_pages)
    _expect_out(pos_offset, "pos_offset", torch.int32, (B,))
    _expect_out(ring_out, "ring_out", torch.int64, (3,))
    _expect_out(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,))
    _expect_out(slots, "slots", torch.int32, (max_tokens,))
    _expect_out(positions, "positions", torch.int32, (max_tokens,))
    dev = _one_device(stream, block_table=block_table, old_lens=old_lens, new_lens=new_lens,
                      free_pages=free_pages, ring=ring, pos_offset=pos_offset, ring_out=ring_out,
                      cu_seqlens=cu_seqlens, slots=slots, positions=positions)
    if ring_out is None:
        ring_out = _new(dev, stream, torch.int64, 3)
    if cu_seqlens is None:
        cu_seqlens = _new(dev, stream, torch.int32, B + 1)
    if slots is None:
        slots = _new(dev, stream, torch.int32, max_tokens)
    if positions is None:
        positions = _new(dev, stream, torch.int32, max_tokens)
    _call(lib().attn_page_update, "attn_page_update", dev, stream, block_table.data_ptr(),
          old_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), ring.data_ptr(),
          ring_out.data_ptr(), cu_seqlens.data_ptr(), slots.data_ptr(), positions.data_ptr(),
          _at(pos_offset), B, max_pages, page_size, num_pages, max_tokens)
    return ring_out, cu_seqlens, slots, positions


def attn_get_device_error(stream=None) -> int:
    """Synchronise the stream, then read and clear the device error flag (0 = none)."""
    return int(lib().attn_get_device_error(_stream_ptr(stream)))


def attn_debug_timeout_probe(limit_cycles: int, stream=None) -> None:
    _raise(lib().attn_debug_timeout_probe(int(limit_cycles), _stream_ptr(stream)),
           "attn_debug_timeout_probe")

"""GB300-native exact attention: FlashAttention-2 forward (dense and packed
varlen, causal or not, with per-row LSE) and split-KV decoding with a
log-sum-exp merge, as hand-written sm_103a kernels behind the C ABI declared in
include/fa.h.

This module is the thin Python binding over libfa.so: the functions named like
the C entry points (``fa_fwd``, ``fa_fwd_varlen``, ``fa_decode_splitkv``,
``fa_splitkv_merge``) only marshal torch CUDA tensors into pointers and sizes
and check the returned status. ``flash_attention``, ``flash_attention_varlen``
and ``flash_decode`` additionally allocate the outputs (and the decode
workspace) with torch. Every step of the computation runs in the library's
kernels; there is no fallback. If libfa.so is missing, the first call raises.

``stream`` (a torch stream or a raw handle) is where a call's work goes; None is
the current stream. The calls that allocate (``flash_*``) behave with a given
stream as under ``torch.cuda.stream(stream)``, behind the work queued so far on
the current stream: outputs belong to that stream's order, and inputs must not
be freed or overwritten before it is done with them.

No call is recorded by autograd, whether or not its inputs require a gradient:
gradients come from the calls named ``*_bwd``.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from typing import NamedTuple

import torch

__all__ = ["FAError", "fa_fwd", "fa_fwd_varlen", "fa_decode_splitkv", "fa_decode_paged_splitkv", "fa_splitkv_merge",
           "fa_decode_splitkv_fused", "fa_decode_paged_splitkv_fused", "fa_bwd", "fa_bwd_workspace_bytes",
           "fa_bwd_varlen", "fa_bwd_varlen_workspace_bytes", "fa_check_device_error", "fa_status_string",
           "fa_test_withhold_load",
           "flash_attention", "flash_attention_varlen", "flash_attention_bwd", "flash_attention_varlen_bwd",
           "fa_fwd_window", "fa_fwd_window_varlen", "fa_bwd_window", "fa_bwd_window_varlen",
           "fa_bwd_window_workspace_bytes", "fa_bwd_window_varlen_workspace_bytes",
           "flash_attention_window", "flash_attention_window_bwd", "flash_attention_window_varlen",
           "flash_attention_window_varlen_bwd",
           "flash_decode", "flash_decode_paged", "fa_kv_write_q4", "fa_kv_read_q4", "fa_decode_paged_window",
           "fa_decode_paged_q4", "fa_decode_splits", "KVCacheQ4", "kv_cache_q4", "flash_kv_write_q4",
           "flash_kv_read_q4", "flash_decode_paged_window", "flash_decode_paged_q4",
           "library_path", "load_library", "EXPORTED_SYMBOLS"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libfa.so")
_lock = threading.Lock()
_lib = None

FA_FP16, FA_BF16 = 0, 1
FA_MAX_SPLITS = 1024
FA_Q4_GROUP = 32
EXPORTED_SYMBOLS = ("fa_fwd", "fa_fwd_varlen", "fa_decode_splitkv", "fa_decode_paged_splitkv", "fa_splitkv_merge",
                    "fa_decode_splitkv_fused", "fa_decode_paged_splitkv_fused", "fa_bwd", "fa_bwd_workspace_bytes",
                    "fa_bwd_varlen", "fa_bwd_varlen_workspace_bytes", "fa_check_device_error", "fa_status_string",
                    "fa_version", "fa_test_withhold_load", "fa_kv_write_q4", "fa_kv_read_q4", "fa_decode_splits",
                    "fa_fwd_window", "fa_fwd_window_varlen", "fa_bwd_window", "fa_bwd_window_varlen",
                    "fa_bwd_window_workspace_bytes", "fa_bwd_window_varlen_workspace_bytes",
                    "fa_decode_paged_window", "fa_decode_paged_q4")


class FAError(RuntimeError):
    """A libfa entry point returned a non-zero status."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


def library_path() -> str:
    return _LIB_PATH


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libfa.so (declares the argument types of every entry point)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is not built: run exact_attention_54_gb300.build.build() "
                               "(or __graft_entry__.build()) first")
        lib = ctypes.CDLL(p)
        vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, vp]
        lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
        lib.fa_decode_splitkv.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        lib.fa_splitkv_merge.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, vp]
        lib.fa_decode_splitkv_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
        lib.fa_decode_paged_splitkv_fused.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i,
                                                      f, i, vp]
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, i, i, i, i, i, i, f, i, vp]
        lib.fa_test_withhold_load.argtypes = [i, ctypes.c_ulonglong]
        lib.fa_bwd.restype = ctypes.c_int
        lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
        lib.fa_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_bwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp, i, i, i, i, i,
                                      i, i, i, f, i, vp]
        lib.fa_bwd_varlen.restype = ctypes.c_int
        lib.fa_bwd_varlen_workspace_bytes.argtypes = [i, i, i]
        lib.fa_bwd_varlen_workspace_bytes.restype = ctypes.c_size_t
        sz = ctypes.c_size_t
        lib.fa_fwd_window.argtypes = [vp] * 5 + [i] * 8 + [f, i, vp]
        lib.fa_fwd_window_varlen.argtypes = [vp] * 7 + [i] * 9 + [f, i, vp]
        lib.fa_bwd_window.argtypes = [vp] * 10 + [sz] + [i] * 8 + [f, i, vp]
        lib.fa_bwd_window_workspace_bytes.argtypes = [i] * 8
        lib.fa_bwd_window_workspace_bytes.restype = sz
        lib.fa_bwd_window_varlen_workspace_bytes.argtypes = [i] * 9
        lib.fa_bwd_window_varlen_workspace_bytes.restype = sz
        lib.fa_bwd_window_varlen.argtypes = [vp] * 10 + [sz, vp, vp] + [i] * 10 + [f, i, vp]
        lib.fa_kv_write_q4.argtypes = [vp] * 9 + [i] * 9 + [vp]
        lib.fa_kv_read_q4.argtypes = [vp] * 9 + [i] * 9 + [vp]
        lib.fa_decode_splits.argtypes = [i, i, i, i]
        lib.fa_decode_paged_window.argtypes = [vp] * 11 + [i] * 10 + [f, i, vp]
        lib.fa_decode_paged_q4.argtypes = [vp] * 13 + [i] * 10 + [f, i, vp]
        lib.fa_check_device_error.argtypes = [vp]
        lib.fa_status_string.argtypes = [i]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_version.argtypes = []
        for name in ("fa_fwd", "fa_fwd_varlen", "fa_decode_splitkv", "fa_splitkv_merge", "fa_decode_splitkv_fused",
                     "fa_decode_paged_splitkv_fused", "fa_check_device_error", "fa_version", "fa_kv_write_q4",
                     "fa_fwd_window", "fa_fwd_window_varlen", "fa_bwd_window", "fa_bwd_window_varlen",
                     "fa_kv_read_q4", "fa_decode_splits", "fa_decode_paged_window", "fa_decode_paged_q4"):
            getattr(lib, name).restype = ctypes.c_int
        if path is None:
            _lib = lib
        return lib


def fa_status_string(status: int) -> str:
    return load_library().fa_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise FAError(fn, status, fa_status_string(status))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return FA_FP16
    if t.dtype == torch.bfloat16:
        return FA_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: expected float16 or bfloat16")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@contextlib.contextmanager
def _on_stream(stream, t):
    """Makes the caller's ``stream`` the current one (of the device of ``t``), behind the work queued so far on the one
    that was. What a call allocates, clears and launches inside is in that stream's order, and so is what the
    allocator does with the memory afterwards."""
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("all tensors must be on one CUDA device")
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream must be one of {dev}, got one of {stream.device}")
    before = torch.cuda.current_stream(dev)
    outside = torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream):
        # (a stream that is being captured cannot wait for one that is not)
        if stream.cuda_stream != before.cuda_stream and (outside or not torch.cuda.is_current_stream_capturing()):
            stream.wait_stream(before)
        yield


def _need_contig(*ts):
    for t in ts:
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


# ------------------------------------------------------------- entry points --

def fa_fwd(q, k, v, o, lse, causal: bool, scale: float | None = None, stream=None):
    """Dense forward: q, o [B,H,Sq,D]; k, v [B,H,Sk,D]; lse [B,H,Sq] fp32."""
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    _need_contig(q, k, v, o, lse)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Sq, Sk, D, int(bool(causal)),
                               float(scale), _dtype_code(q), _stream(stream))
    _check("fa_fwd", st)


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, causal: bool,
                  scale: float | None = None, stream=None):
    """Packed forward: q, o [total_q,H,D]; k, v [total_k,H,D]; lse [H,total_q];
    cu_seqlens_* int32 CUDA tensors of length num_seqs+1."""
    Tq, H, D = q.shape
    Tk = k.shape[0]
    _need_contig(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q),
                                      _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, Tq, Tk, int(max_seqlen_q), H,
                                      D, int(bool(causal)), float(scale), _dtype_code(q), _stream(stream))
    _check("fa_fwd_varlen", st)


def fa_decode_splitkv(q, k, v, o_part, m_part, l_part, num_splits: int, scale: float | None = None, stream=None):
    """Phase 1: q [B,H,1,D] (or [B,H,D]); k, v [B,H,Sk,D]; o_part [B,H,S,D],
    m_part and l_part [B,H,S] fp32."""
    B, H, Sk, D = k.shape
    _need_contig(q, k, v, o_part, m_part, l_part)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_decode_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o_part), _ptr(m_part), _ptr(l_part),
                                          B, H, Sk, D, int(num_splits), float(scale), _dtype_code(k),
                                          _stream(stream))
    _check("fa_decode_splitkv", st)


def fa_decode_paged_splitkv(q, k_cache, v_cache, block_table, seq_lens, o_part, m_part, l_part, num_splits: int,
                            scale: float | None = None, stream=None):
    """Phase 1 over a paged cache: q [B,H,1,D]; k_cache, v_cache
    [num_blocks,H,block_size,D]; block_table [B,max_blocks] and seq_lens [B]
    int32 CUDA tensors; partials as in fa_decode_splitkv."""
    B, H = q.shape[0], q.shape[1]
    num_blocks, _, block_size, D = k_cache.shape
    _need_contig(q, k_cache, v_cache, block_table, seq_lens, o_part, m_part, l_part)
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    lib = load_library()
    fn = lib.fa_decode_paged_splitkv
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
    fn.restype = ctypes.c_int
    _check("fa_decode_paged_splitkv",
           fn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens), _ptr(o_part), _ptr(m_part),
              _ptr(l_part), B, H, D, num_blocks, block_size, block_table.shape[1], int(num_splits), float(scale),
              _dtype_code(q), _stream(stream)))


def fa_splitkv_merge(o_part, m_part, l_part, o, lse, stream=None):
    """Phase 2: partials from phase 1 -> o [B,H,1,D] (16-bit), lse [B,H] fp32."""
    B, H, S, D = o_part.shape
    _need_contig(o_part, m_part, l_part, o, lse)
    st = load_library().fa_splitkv_merge(_ptr(o_part), _ptr(m_part), _ptr(l_part), _ptr(o), _ptr(lse), B, H, D,
                                         S, _dtype_code(o), _stream(stream))
    _check("fa_splitkv_merge", st)


def fa_decode_splitkv_fused(q, k, v, o, lse, o_part, m_part, l_part, counters, num_splits: int,
                            scale: float | None = None, stream=None):
    """Both decode phases in one launch. Arguments as fa_decode_splitkv plus
    o [B,H,1,D], lse [B,H] and counters, an int32 [B*H] CUDA tensor that is
    zero before the first call and is left zero by every completed call."""
    B, H, Sk, D = k.shape
    _need_contig(q, k, v, o, lse, o_part, m_part, l_part, counters)
    if counters.dtype != torch.int32:
        raise TypeError("counters must be int32")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_decode_splitkv_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(o_part),
                                                _ptr(m_part), _ptr(l_part), _ptr(counters), B, H, Sk, D,
                                                int(num_splits), float(scale), _dtype_code(k), _stream(stream))
    _check("fa_decode_splitkv_fused", st)


def fa_decode_paged_splitkv_fused(q, k_cache, v_cache, block_table, seq_lens, o, lse, o_part, m_part, l_part,
                                  counters, num_splits: int, scale: float | None = None, stream=None):
    """Both decode phases over a paged cache in one launch (arguments as
    fa_decode_paged_splitkv plus o, lse and counters as fa_decode_splitkv_fused)."""
    B, H = q.shape[0], q.shape[1]
    num_blocks, _, block_size, D = k_cache.shape
    _need_contig(q, k_cache, v_cache, block_table, seq_lens, o, lse, o_part, m_part, l_part, counters)
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or counters.dtype != torch.int32:
        raise TypeError("block_table, seq_lens and counters must be int32")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_decode_paged_splitkv_fused(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens), _ptr(o), _ptr(lse), _ptr(o_part),
        _ptr(m_part), _ptr(l_part), _ptr(counters), B, H, D, num_blocks, block_size, block_table.shape[1],
        int(num_splits), float(scale), _dtype_code(q), _stream(stream))
    _check("fa_decode_paged_splitkv_fused", st)


def fa_bwd_workspace_bytes(B: int, H: int, Sq: int, D: int) -> int:
    return int(load_library().fa_bwd_workspace_bytes(B, H, Sq, D))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal: bool, scale: float | None = None, stream=None):
    """Backward pass: q, o, dout, dq [B,H,Sq,D]; k, v, dk, dv [B,H,Sk,D];
    lse [B,H,Sq] fp32 from the forward; workspace a CUDA tensor of at least
    fa_bwd_workspace_bytes(B, H, Sq, D) bytes."""
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    _need_contig(q, k, v, o, dout, lse, dq, dk, dv, workspace)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(), B, H, Sq,
                               Sk, D, int(bool(causal)), float(scale), _dtype_code(q), _stream(stream))
    _check("fa_bwd", st)


def fa_bwd_varlen_workspace_bytes(total_q: int, H: int, D: int) -> int:
    return int(load_library().fa_bwd_varlen_workspace_bytes(total_q, H, D))


def fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                  max_seqlen_k: int, causal: bool, scale: float | None = None, stream=None):
    """Backward pass over packed sequences: q, o, dout, dq [total_q,H,D]; k, v,
    dk, dv [total_k,H,D]; lse [H,total_q] fp32 from fa_fwd_varlen;
    cu_seqlens_* int32 CUDA tensors of length num_seqs+1; workspace a CUDA
    tensor of at least fa_bwd_varlen_workspace_bytes(total_q, H, D) bytes."""
    Tq, H, D = q.shape
    Tk = k.shape[0]
    _need_contig(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k)
    if cu_seqlens_q.dtype != torch.int32 or cu_seqlens_k.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    st = load_library().fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk),
                                      _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, Tq, Tk,
                                      int(max_seqlen_q), int(max_seqlen_k), H, D, int(bool(causal)), float(scale),
                                      _dtype_code(q), _stream(stream))
    _check("fa_bwd_varlen", st)


def fa_test_withhold_load(load: int, wait_limit_ns: int = 0):
    """Test support: make the CTA with the first work item of later prefill
    launches withhold one tile load so that their bounded wait runs out (see include/fa.h); (0, 0) turns
    it off."""
    _check("fa_test_withhold_load", load_library().fa_test_withhold_load(int(load), int(wait_limit_ns)))


def fa_check_device_error(stream=None):
    """Synchronise the stream and raise if a kernel abandoned a barrier wait."""
    _check("fa_check_device_error", load_library().fa_check_device_error(_stream(stream)))


# ------------------------------------------------------ allocating helpers --

def _words(n: int) -> int:
    """fp32 elements of a workspace of n bytes; one where n is 0, so that a call with sizes that the library refuses
    gets that refusal and not one of a NULL pointer."""
    return max(n // 4, 1)


def flash_attention(q, k, v, causal: bool = False, scale: float | None = None, stream=None):
    """Returns (o, lse) for dense [B,H,S,D] CUDA tensors."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention(q, k, v, causal, scale)
    B, H, Sq, D = q.shape
    o = torch.empty_like(q)
    lse = torch.empty(B, H, Sq, dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, causal, scale)
    return o, lse


def flash_attention_bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, stream=None,
                        workspace=None):
    """Returns (dq, dk, dv) for dense [B,H,S,D] CUDA tensors, given the
    forward's o and lse."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_bwd(q, k, v, o, lse, dout, causal, scale, workspace=workspace)
    B, H, Sq, D = q.shape
    if workspace is None:
        workspace = torch.empty(_words(fa_bwd_workspace_bytes(B, H, Sq, D)), dtype=torch.float32, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, workspace, causal, scale)
    return dq, dk, dv


def flash_attention_varlen_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                               max_seqlen_k: int, causal: bool = False, scale: float | None = None, stream=None,
                               workspace=None):
    """Returns (dq, dk, dv) for packed sequences, given fa_fwd_varlen's o and lse."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_varlen_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                                              max_seqlen_k, causal, scale, workspace=workspace)
    Tq, H, D = q.shape
    if workspace is None:
        workspace = torch.empty(_words(fa_bwd_varlen_workspace_bytes(Tq, H, D)), dtype=torch.float32, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                  max_seqlen_k, causal, scale)
    return dq, dk, dv


def flash_attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, causal: bool = False,
                           scale: float | None = None, stream=None):
    """Returns (o [total_q,H,D], lse [H,total_q]) for packed sequences."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal, scale)
    Tq, H, D = q.shape
    o = torch.empty_like(q)
    lse = torch.empty(H, Tq, dtype=torch.float32, device=q.device)
    fa_fwd_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, causal, scale)
    return o, lse


def _decode_workspace(B, H, S, D, device, fused):
    ws = (torch.empty(B, H, S, D, dtype=torch.float32, device=device),
          torch.empty(B, H, S, dtype=torch.float32, device=device),
          torch.empty(B, H, S, dtype=torch.float32, device=device))
    return ws + (torch.zeros(B * H, dtype=torch.int32, device=device),) if fused else ws


def flash_decode_paged(q, k_cache, v_cache, block_table, seq_lens, num_splits: int, scale: float | None = None,
                       stream=None, workspace=None, fused: bool = False):
    """Split-KV decoding over a paged cache (phase 1 + phase 2). Returns
    (o [B,H,1,D], lse [B,H]). ``workspace`` may pass preallocated (o_part,
    m_part, l_part), plus the int32 [B*H] counters when ``fused``."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_decode_paged(q, k_cache, v_cache, block_table, seq_lens, num_splits, scale,
                                      workspace=workspace, fused=fused)
    B, H = q.shape[0], q.shape[1]
    D = k_cache.shape[3]
    if workspace is None:
        workspace = _decode_workspace(B, H, num_splits, D, q.device, fused)
    o = torch.empty(B, H, 1, D, dtype=q.dtype, device=q.device)
    lse = torch.empty(B, H, dtype=torch.float32, device=q.device)
    if fused:
        fa_decode_paged_splitkv_fused(q, k_cache, v_cache, block_table, seq_lens, o, lse, *workspace, num_splits,
                                      scale)
        return o, lse
    o_part, m_part, l_part = workspace[:3]
    fa_decode_paged_splitkv(q, k_cache, v_cache, block_table, seq_lens, o_part, m_part, l_part, num_splits, scale)
    fa_splitkv_merge(o_part, m_part, l_part, o, lse)
    return o, lse


def flash_decode(q, k, v, num_splits: int, scale: float | None = None, stream=None, workspace=None,
                 fused: bool = False):
    """Split-KV decoding (phase 1 + phase 2). Returns (o [B,H,1,D], lse [B,H]).
    ``workspace`` may pass preallocated (o_part, m_part, l_part), plus the
    int32 [B*H] counters when ``fused`` (one launch instead of two)."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_decode(q, k, v, num_splits, scale, workspace=workspace, fused=fused)
    B, H, Sk, D = k.shape
    if workspace is None:
        workspace = _decode_workspace(B, H, num_splits, D, k.device, fused)
    o = torch.empty(B, H, 1, D, dtype=k.dtype, device=k.device)
    lse = torch.empty(B, H, dtype=torch.float32, device=k.device)
    if fused:
        fa_decode_splitkv_fused(q, k, v, o, lse, *workspace, num_splits, scale)
        return o, lse
    o_part, m_part, l_part = workspace[:3]
    fa_decode_splitkv(q, k, v, o_part, m_part, l_part, num_splits, scale)
    fa_splitkv_merge(o_part, m_part, l_part, o, lse)
    return o, lse


def fa_decode_noalloc(q, k, v, o, lse, num_splits: int, scale: float | None = None, stream=None):
    """Split-KV decoding (both phases) with no device allocation and no
    workspace argument, for callers that cannot allocate device memory when
    they call in. The partials use a fixed device array built into the
    library (FA_NOALLOC_SCRATCH_FLOATS floats); concurrent calls whose GPU work
    overlaps race on it. q [B,H,1,D]; k, v [B,H,Sk,D]; o [B,H,1,D]; lse [B,H]."""
    lib = load_library()
    fn = lib.fa_decode_noalloc
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    fn.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    fn.restype = ctypes.c_int
    B, H, Sk, D = k.shape
    _need_contig(q, k, v, o, lse)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    _check("fa_decode_noalloc", fn(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Sk, D, int(num_splits),
                                   float(scale), _dtype_code(k), _stream(stream)))


# ------------------------------------- shared key heads, windows, 4-bit cache --

def _int32(n) -> int:
    """A whole number as a C int, the nearest one where it does not fit (ctypes would drop its upper bits)."""
    n = int(n)
    return n if -0x80000000 <= n <= 0x7fffffff else 0x7fffffff if n > 0 else -0x80000000


def _expect(name: str, t, shape, dtype):
    """Refuse a tensor that is not a contiguous one of this shape and dtype (None in ``shape``: any size)."""
    if t.dtype == dtype and t.shape == shape and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_entry = {}  # entry points of the loaded library by name
# handle of a device's current stream, without a Stream object where PyTorch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(fn: str, stream, tensors, *args, index=None):
    """Call entry point ``fn`` with the pointers of ``tensors`` (None: NULL), ``args`` and the stream, on the device
    that the tensors, and those of ``index``, share."""
    dev = tensors[0].get_device()
    ptrs = []
    for t in tensors:
        if t is None:
            ptrs.append(None)
        elif t.get_device() == dev:
            ptrs.append(t.data_ptr())
        else:
            dev = -1
    for t in index or ():
        if t.get_device() != dev:
            dev = -1
    if dev < 0:
        raise ValueError(f"{fn}: all tensors must be on one CUDA device")
    call = _entry.get(fn)
    if call is None:
        call = _entry[fn] = getattr(load_library(), fn)
    stream = _raw_stream(dev) if stream is None else _stream(stream)
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            st = call(*ptrs, *args, stream)
    else:
        st = call(*ptrs, *args, stream)
    if st != 0:
        _check(fn, st)


def fa_fwd_window(q, k, v, o, lse, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """Causal attention with a sliding window and sinks: q, o [B,H,Sq,D]; k, v [B,Hkv,Sk,D]; lse [B,H,Sq] fp32."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,Sq,D] and k, v [B,Hkv,Sk,D]")
    B, H, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    code = _dtype_code(q)
    for name, t, shape in (("q", q, (B, H, Sq, D)), ("k", k, (B, Hkv, Sk, D)), ("v", v, (B, Hkv, Sk, D)),
                           ("o", o, (B, H, Sq, D))):
        _expect(name, t, shape, q.dtype)
    _expect("lse", lse, (B, H, Sq), torch.float32)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ts = (q, k, v, o, lse)
    _launch("fa_fwd_window", stream, ts, B, H, Hkv, Sq, Sk, D, _int32(window), _int32(sinks), float(scale), code)


def fa_fwd_window_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, window: int, sinks: int = 0,
                         scale: float | None = None, stream=None):
    """fa_fwd_window over packed sequences: q, o [total_q,H,D]; k, v [total_k,Hkv,D]; lse [H,total_q]."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [total_q,H,D] and k, v [total_k,Hkv,D]")
    Tq, H, D = q.shape
    Tk, Hkv, _ = k.shape
    n = cu_seqlens_q.numel() - 1
    code = _dtype_code(q)
    for name, t, shape in (("q", q, (Tq, H, D)), ("k", k, (Tk, Hkv, D)), ("v", v, (Tk, Hkv, D)), ("o", o, (Tq, H, D))):
        _expect(name, t, shape, q.dtype)
    _expect("lse", lse, (H, Tq), torch.float32)
    _expect("cu_seqlens_q", cu_seqlens_q, (n + 1,), torch.int32)
    _expect("cu_seqlens_k", cu_seqlens_k, (n + 1,), torch.int32)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ts = (q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
    _launch("fa_fwd_window_varlen", stream, ts, n, Tq, Tk, _int32(max_seqlen_q), H, Hkv, D, _int32(window),
            _int32(sinks), float(scale), code)


def fa_bwd_window_workspace_bytes(B: int, H: int, Hkv: int, Sq: int, Sk: int, D: int, window: int,
                                  sinks: int = 0) -> int:
    return int(load_library().fa_bwd_window_workspace_bytes(*map(_int32, (B, H, Hkv, Sq, Sk, D, window, sinks))))


def fa_bwd_window_varlen_workspace_bytes(num_seqs: int, total_q: int, max_seqlen_q: int, max_seqlen_k: int, H: int,
                                         Hkv: int, D: int, window: int, sinks: int = 0) -> int:
    args = (num_seqs, total_q, max_seqlen_q, max_seqlen_k, H, Hkv, D, window, sinks)
    return int(load_library().fa_bwd_window_varlen_workspace_bytes(*map(_int32, args)))


def fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, window: int, sinks: int = 0,
                  scale: float | None = None, stream=None):
    """Gradients of fa_fwd_window: q, o, dout, dq [B,H,Sq,D]; k, v, dk, dv [B,Hkv,Sk,D]; workspace of at least
    fa_bwd_window_workspace_bytes(B, H, Hkv, Sq, Sk, D, window, sinks) bytes."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B,H,Sq,D] and k, v [B,Hkv,Sk,D]")
    B, H, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    code = _dtype_code(q)
    for name, t in (("q", q), ("o", o), ("dout", dout), ("dq", dq)):
        _expect(name, t, (B, H, Sq, D), q.dtype)
    for name, t in (("k", k), ("v", v), ("dk", dk), ("dv", dv)):
        _expect(name, t, (B, Hkv, Sk, D), q.dtype)
    _expect("lse", lse, (B, H, Sq), torch.float32)
    _need_contig(workspace)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ts = (q, k, v, o, dout, lse, dq, dk, dv, workspace)
    _launch("fa_bwd_window", stream, ts, workspace.numel() * workspace.element_size(), B, H, Hkv, Sq, Sk, D,
            _int32(window), _int32(sinks), float(scale), code)


def fa_bwd_window_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                         max_seqlen_k: int, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """Gradients of fa_fwd_window_varlen: q, o, dout, dq [total_q,H,D]; k, v, dk, dv [total_k,Hkv,D]; workspace of at
    least fa_bwd_window_varlen_workspace_bytes bytes."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [total_q,H,D] and k, v [total_k,Hkv,D]")
    Tq, H, D = q.shape
    Tk, Hkv, _ = k.shape
    n = cu_seqlens_q.numel() - 1
    code = _dtype_code(q)
    for name, t in (("q", q), ("o", o), ("dout", dout), ("dq", dq)):
        _expect(name, t, (Tq, H, D), q.dtype)
    for name, t in (("k", k), ("v", v), ("dk", dk), ("dv", dv)):
        _expect(name, t, (Tk, Hkv, D), q.dtype)
    _expect("lse", lse, (H, Tq), torch.float32)
    _expect("cu_seqlens_q", cu_seqlens_q, (n + 1,), torch.int32)
    _expect("cu_seqlens_k", cu_seqlens_k, (n + 1,), torch.int32)
    _need_contig(workspace)
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    ts = (q, k, v, o, dout, lse, dq, dk, dv, workspace)
    _launch("fa_bwd_window_varlen", stream, ts, workspace.numel() * workspace.element_size(), cu_seqlens_q.data_ptr(),
            cu_seqlens_k.data_ptr(), n, Tq, Tk, _int32(max_seqlen_q), _int32(max_seqlen_k), H, Hkv, D, _int32(window),
            _int32(sinks), float(scale), code, index=(cu_seqlens_q, cu_seqlens_k))


def flash_attention_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """Returns (o, lse) of causal attention with a sliding window and sinks: q [B,H,Sq,D], k, v [B,Hkv,Sk,D]. Not
    recorded by autograd: flash_attention_window_bwd gives the gradients."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_window(q, k, v, window, sinks, scale)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    fa_fwd_window(q, k, v, o, lse, window, sinks, scale)
    return o, lse


def flash_attention_window_bwd(q, k, v, o, lse, dout, window: int, sinks: int = 0, scale: float | None = None,
                               stream=None, workspace=None):
    """Returns (dq, dk, dv) of flash_attention_window, given its o and lse."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_window_bwd(q, k, v, o, lse, dout, window, sinks, scale, workspace=workspace)
    if workspace is None:
        if q.dim() != 4 or k.dim() != 4:
            raise ValueError("q must be [B,H,Sq,D] and k, v [B,Hkv,Sk,D]")
        (B, H, Sq, D), (_, Hkv, Sk, _) = q.shape, k.shape
        workspace = torch.empty(_words(fa_bwd_window_workspace_bytes(B, H, Hkv, Sq, Sk, D, window, sinks)),
                                dtype=torch.float32, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, workspace, window, sinks, scale)
    return dq, dk, dv


def flash_attention_window_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int, window: int, sinks: int = 0,
                                  scale: float | None = None, stream=None):
    """Returns (o [total_q,H,D], lse [H,total_q]) for packed sequences; k, v [total_k,Hkv,D]."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_window_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, window, sinks,
                                                 scale)
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[1], q.shape[0], dtype=torch.float32, device=q.device)
    fa_fwd_window_varlen(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, window, sinks, scale)
    return o, lse


def flash_attention_window_varlen_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                                      max_seqlen_k: int, window: int, sinks: int = 0, scale: float | None = None,
                                      stream=None, workspace=None):
    """Returns (dq, dk, dv) of flash_attention_window_varlen, given its o and lse."""
    if stream is not None:
        with _on_stream(stream, q):
            return flash_attention_window_varlen_bwd(q, k, v, o, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                                                     max_seqlen_k, window, sinks, scale, workspace=workspace)
    if workspace is None:
        if q.dim() != 3 or k.dim() != 3:
            raise ValueError("q must be [total_q,H,D] and k, v [total_k,Hkv,D]")
        Tq, H, D = q.shape
        n = fa_bwd_window_varlen_workspace_bytes(cu_seqlens_q.numel() - 1, Tq, max_seqlen_q, max_seqlen_k, H,
                                                 k.shape[1], D, window, sinks)
        workspace = torch.empty(_words(n), dtype=torch.float32, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    fa_bwd_window_varlen(q, k, v, o, dout, lse, dq, dk, dv, workspace, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, window, sinks, scale)
    return dq, dk, dv


class KVCacheQ4(NamedTuple):
    """The paged 4-bit cache of include/fa.h: codes uint8 [num_blocks,Hkv,block_size,D/2] and scales (fp16 or
    bf16) [num_blocks,Hkv,block_size,D/32] of keys and of values."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def kv_cache_q4(num_blocks: int, Hkv: int, block_size: int, D: int, dtype=torch.bfloat16, device="cuda") -> KVCacheQ4:
    """An empty 4-bit cache (all zeros: rows that were never written read as zero)."""
    rows = (num_blocks, Hkv, block_size)
    one = lambda: (torch.zeros(*rows, D // 2, dtype=torch.uint8, device=device),  # noqa: E731
                   torch.zeros(*rows, D // FA_Q4_GROUP, dtype=dtype, device=device))
    return KVCacheQ4(*one(), *one())


def _check_q4(k_codes, k_scales, v_codes, v_scales, Hkv, D, dtype):
    num_blocks, block_size = (k_codes.shape[0], k_codes.shape[2]) if k_codes.dim() == 4 else (None, None)
    codes, scales = (num_blocks, Hkv, block_size, D // 2), (num_blocks, Hkv, block_size, D // FA_Q4_GROUP)
    _expect("k_codes", k_codes, codes, torch.uint8)
    _expect("v_codes", v_codes, codes, torch.uint8)
    _expect("k_scales", k_scales, scales, dtype)
    _expect("v_scales", v_scales, scales, dtype)
    return num_blocks, block_size


def _kv_q4(fn, k, v, cache, block_table, cu_seqlens, max_seqlen, starts, stream):
    if k.dim() != 3:
        raise ValueError(f"k must be [total,Hkv,D], got {tuple(k.shape)}")
    total, Hkv, D = k.shape
    code = _dtype_code(k)
    _expect("k", k, (total, Hkv, D), k.dtype)
    _expect("v", v, (total, Hkv, D), k.dtype)
    num_blocks, block_size = _check_q4(*cache, Hkv, D, k.dtype)
    n = cu_seqlens.numel() - 1
    _expect("cu_seqlens", cu_seqlens, (n + 1,), torch.int32)
    _expect("block_table", block_table, (n, block_table.shape[-1]), torch.int32)
    if starts is not None:
        _expect("starts", starts, (n,), torch.int32)
    _launch(fn, stream, (k, v, *cache, block_table, cu_seqlens, starts), n, total, _int32(max_seqlen), Hkv, D,
            num_blocks, block_size, block_table.shape[1], code)


def fa_kv_write_q4(k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, max_seqlen: int, starts=None,
                   stream=None):
    """Quantise the new tokens' k, v [total,Hkv,D] and store them at positions starts[b].. (zero when None) of their
    sequences; cu_seqlens int32 [num_seqs+1], block_table int32 [num_seqs,max_blocks], starts int32 [num_seqs]."""
    _kv_q4("fa_kv_write_q4", k, v, (k_codes, k_scales, v_codes, v_scales), block_table, cu_seqlens, max_seqlen, starts,
           stream)


def fa_kv_read_q4(k, v, k_codes, k_scales, v_codes, v_scales, block_table, cu_seqlens, max_seqlen: int, starts=None,
                  stream=None):
    """Read positions starts[b].. of each sequence back into k, v [total,Hkv,D] (arguments as fa_kv_write_q4)."""
    _kv_q4("fa_kv_read_q4", k, v, (k_codes, k_scales, v_codes, v_scales), block_table, cu_seqlens, max_seqlen, starts,
           stream)


def fa_decode_splits(B: int, H: int, Hkv: int, max_keys: int) -> int:
    """A num_splits that is fast on the current GPU (see include/fa.h)."""
    call = _entry.get("fa_decode_splits")
    if call is None:
        call = _entry["fa_decode_splits"] = load_library().fa_decode_splits
    return call(B, H, Hkv, _int32(max_keys))


def _decode_gqa(q, cache, block_table, seq_lens, o, lse, o_part, m_part, l_part, counters, num_splits, window, sinks,
                scale, stream):
    if q.dim() != 4 or cache[0].dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [B,H,1,D], pages 4-dimensional and block_table [B,max_blocks]")
    B, H, _, D = q.shape
    num_blocks, Hkv, block_size, _ = cache[0].shape
    code = _dtype_code(q)
    if len(cache) == 4:
        fn = "fa_decode_paged_q4"
        _check_q4(*cache, Hkv, D, q.dtype)
    else:
        fn = "fa_decode_paged_window"
        _expect("k_cache", cache[0], (num_blocks, Hkv, block_size, D), q.dtype)
        _expect("v_cache", cache[1], (num_blocks, Hkv, block_size, D), q.dtype)
    max_blocks = block_table.shape[1]
    _expect("q", q, (B, H, 1, D), q.dtype)
    _expect("block_table", block_table, (B, max_blocks), torch.int32)
    _expect("seq_lens", seq_lens, (B,), torch.int32)
    _expect("o", o, (B, H, 1, D), q.dtype)
    _expect("lse", lse, (B, H), torch.float32)
    S = _int32(num_splits)
    rows = B * H * S
    for name, t, need, dtype in (("o_part", o_part, rows * D, torch.float32), ("m_part", m_part, rows, torch.float32),
                                 ("l_part", l_part, rows, torch.float32), ("counters", counters, B * H, torch.int32)):
        if t.numel() < need or t.dtype != dtype or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous {dtype} of at least {need} elements")
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    _launch(fn, stream, (q, *cache, block_table, seq_lens, o, lse, o_part, m_part, l_part, counters), B, H, Hkv, D,
            num_blocks, block_size, max_blocks, S, _int32(window), _int32(sinks), float(scale), code)


def fa_decode_paged_window(q, k_cache, v_cache, block_table, seq_lens, o, lse, o_part, m_part, l_part, counters,
                           num_splits: int, window: int, sinks: int = 0, scale: float | None = None, stream=None):
    """One-token attention over a paged cache: q [B,H,1,D]; k_cache, v_cache [num_blocks,Hkv,block_size,D]; the token
    sees its last ``window`` keys (0: all) and the first ``sinks``. o_part [B,H,num_splits,D], m_part and l_part
    [B,H,num_splits] fp32 and counters int32 [B*H] (zero between calls) may be larger than that."""
    _decode_gqa(q, (k_cache, v_cache), block_table, seq_lens, o, lse, o_part, m_part, l_part, counters, num_splits,
                window, sinks, scale, stream)


def fa_decode_paged_q4(q, k_codes, k_scales, v_codes, v_scales, block_table, seq_lens, o, lse, o_part, m_part, l_part,
                       counters, num_splits: int, window: int = 0, sinks: int = 0, scale: float | None = None,
                       stream=None):
    """fa_decode_paged_window over the 4-bit cache (scales in the dtype of q)."""
    _decode_gqa(q, (k_codes, k_scales, v_codes, v_scales), block_table, seq_lens, o, lse, o_part, m_part, l_part,
                counters, num_splits, window, sinks, scale, stream)


def flash_kv_write_q4(k, v, cache: KVCacheQ4, block_table, cu_seqlens, max_seqlen: int, starts=None, stream=None):
    """fa_kv_write_q4 into the four tensors of ``cache``."""
    _kv_q4("fa_kv_write_q4", k, v, cache, block_table, cu_seqlens, max_seqlen, starts, stream)


def flash_kv_read_q4(cache: KVCacheQ4, block_table, cu_seqlens, total: int, max_seqlen: int, starts=None, stream=None):
    """Returns (k, v) [total,Hkv,D] with positions starts[b].. of each sequence, packed by cu_seqlens. Rows that belong
    to no sequence (total above cu_seqlens[-1]) are not initialised: flash_attention_window_varlen takes no notice of
    them, for flash_attention_varlen they have to be cleared."""
    if stream is not None:
        with _on_stream(stream, cache[0]):
            return flash_kv_read_q4(cache, block_table, cu_seqlens, total, max_seqlen, starts)
    codes, scales = cache[0], cache[1]
    k = torch.empty(int(total), codes.shape[1], 2 * codes.shape[3], dtype=scales.dtype, device=codes.device)
    v = torch.empty_like(k)
    _kv_q4("fa_kv_read_q4", k, v, cache, block_table, cu_seqlens, max_seqlen, starts, None)
    return k, v


def _flash_decode_gqa(q, cache, block_table, seq_lens, window, sinks, num_splits, scale, stream, workspace):
    if stream is not None:
        with _on_stream(stream, q):
            return _flash_decode_gqa(q, cache, block_table, seq_lens, window, sinks, num_splits, scale, None, workspace)
    if q.dim() != 4 or cache[0].dim() != 4 or block_table.dim() != 2:
        raise ValueError("q must be [B,H,1,D], pages 4-dimensional and block_table [B,max_blocks]")
    B, H, _, D = q.shape
    _, Hkv, block_size, _ = cache[0].shape
    if num_splits is None:
        keys = block_table.shape[1] * block_size
        if window > 0:
            keys = min(keys, window + sinks)
        num_splits = fa_decode_splits(B, H, Hkv, keys)
        if workspace is not None:
            num_splits = min(num_splits, workspace[1].numel() // max(B * H, 1))
    if workspace is None:
        workspace = _decode_workspace(B, H, num_splits, D, q.device, True)
    o, lse = torch.empty_like(q), torch.empty((B, H), dtype=torch.float32, device=q.device)
    _decode_gqa(q, cache, block_table, seq_lens, o, lse, *workspace, num_splits, window, sinks, scale, None)
    return o, lse


def flash_decode_paged_window(q, k_cache, v_cache, block_table, seq_lens, window: int, sinks: int = 0,
                              num_splits: int | None = None, scale: float | None = None, stream=None, workspace=None):
    """One-token attention over a paged cache with shared key heads, a sliding window (0: none) and sinks. Returns
    (o [B,H,1,D], lse [B,H]). ``workspace`` may pass (o_part, m_part, l_part, counters), counters zero; num_splits
    None takes fa_decode_splits, within the workspace."""
    return _flash_decode_gqa(q, (k_cache, v_cache), block_table, seq_lens, window, sinks,
                             num_splits, scale, stream, workspace)


def flash_decode_paged_q4(q, cache: KVCacheQ4, block_table, seq_lens, window: int = 0, sinks: int = 0,
                          num_splits: int | None = None, scale: float | None = None, stream=None, workspace=None):
    """flash_decode_paged_window over the 4-bit cache."""
    return _flash_decode_gqa(q, tuple(cache), block_table, seq_lens, window, sinks, num_splits, scale, stream,
                             workspace)

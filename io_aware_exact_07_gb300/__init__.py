"""Exact IO-aware attention (forward + backward) for GB300 / sm_103a.

Thin ctypes binding over the C ABI in ``include/fa.h`` (libfa_gb300.so, built
in-tree by ``io_aware_exact_07_gb300.build``). Functions named ``fa_*`` mirror
the C entry points one to one and only marshal arguments (torch tensors ->
device pointers, the current torch CUDA stream); every step of the
computation runs in the library's CUDA kernels. There is no CPU fallback: if
the library is missing or fails to load, calls raise.

``fwd`` / ``bwd`` are conveniences that allocate the outputs (and the backward
workspace) with torch and call ``fa_fwd`` / ``fa_bwd``; ``decode`` does the
same for ``fa_decode`` (short query blocks over a K/V cache). ``paged_write``,
``paged_read`` and ``paged_attn`` work on a cache held in pages, in bf16 or
quantised to e4m3 (``paged_cache`` allocates one).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_WORKSPACE = 4
FA_ERR_TIMEOUT = 5

FA_CACHE_BF16 = 0
FA_CACHE_E4M3 = 1

# Symbols declared in include/fa.h.
EXPORTS = (
    "fa_fwd", "fa_bwd", "fa_fwd_gqa", "fa_bwd_gqa", "fa_fwd_window", "fa_bwd_window",
    "fa_bwd_workspace_size", "fa_bwd_preprocess",
    "fa_bwd_dkdv", "fa_bwd_dq", "fa_decode", "fa_decode_workspace_size",
    "fa_paged_write", "fa_paged_read", "fa_paged_attn", "fa_paged_workspace_size",
    "fa_paged_write_block", "fa_paged_read_block", "fa_paged_attn_block",
    "fa_fp8_workspace_size", "fa_fp8_vt_stride", "fa_fp8_quantize", "fa_fwd_fp8",
    "fa_fp8_quantize_gqa", "fa_fwd_fp8_gqa",
    "fa_bwd_noalloc", "fa_dropout_p8", "fa_debug_dropout_keep",
    "fa_debug_philox", "fa_butterfly_mask", "fa_device_status", "fa_set_wait_timeout_ns",
    "fa_test_inject_stall", "fa_status_string",
)

_lock = threading.Lock()
_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load(build_if_missing: bool = False):
    """Load libfa_gb300.so (optionally building it first). Raises if unavailable."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_missing or not os.path.exists(LIB_PATH):
            if not build_if_missing:
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m io_aware_exact_07_gb300.build`")
            from . import build as _b
            _b.build()
        lib = ctypes.CDLL(LIB_PATH)
        vp, i, f, u64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64,
                             ctypes.c_size_t)
        lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u64, vp, vp, vp]
        lib.fa_fwd.restype = i
        lib.fa_bwd_workspace_size.argtypes = [i, i, i, i]
        lib.fa_bwd_workspace_size.restype = sz
        lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u64,
                               vp, vp, vp, sz, vp]
        lib.fa_bwd.restype = i
        lib.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, u64, u64, vp, vp,
                                   vp]
        lib.fa_fwd_gqa.restype = i
        lib.fa_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, f, u64,
                                   u64, vp, vp, vp, sz, vp]
        lib.fa_bwd_gqa.restype = i
        lib.fa_fwd_window.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, f, u64, u64,
                                      vp, vp, vp]
        lib.fa_fwd_window.restype = i
        lib.fa_bwd_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, i,
                                      f, u64, u64, vp, vp, vp, sz, vp]
        lib.fa_bwd_window.restype = i
        lib.fa_bwd_preprocess.argtypes = [vp, vp, i, i, i, i, vp, sz, vp]
        lib.fa_bwd_preprocess.restype = i
        lib.fa_bwd_dkdv.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u64, vp,
                                    vp, vp, sz, vp]
        lib.fa_bwd_dkdv.restype = i
        lib.fa_bwd_dq.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f, u64, u64, vp, vp,
                                  vp, sz, vp]
        lib.fa_bwd_dq.restype = i
        lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, f,
                                       u64, u64, vp, vp, vp]
        lib.fa_bwd_noalloc.restype = i
        lib.fa_decode_workspace_size.argtypes = [i, i, i, i, i, i, i]
        lib.fa_decode_workspace_size.restype = sz
        lib.fa_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, i, vp, i, vp, sz, vp]
        lib.fa_decode.restype = i
        i64 = ctypes.c_int64
        cache = [i, i, i, i, i, i64, i64, i64, vp, i64, i, vp]  # type .. d, strides, table, lengths
        lib.fa_paged_write.argtypes = [vp] * 6 + cache + [vp, i, i, i, i64, i64, vp]
        lib.fa_paged_write.restype = i
        lib.fa_paged_read.argtypes = [vp] * 4 + cache + [i, i, vp, vp, vp]
        lib.fa_paged_read.restype = i
        for f_block in (lib.fa_paged_write_block, lib.fa_paged_read_block, lib.fa_paged_attn_block):
            f_block.argtypes = [ctypes.c_char_p, vp]
            f_block.restype = i
        lib.fa_paged_workspace_size.argtypes = [i, i, i, i, i]
        lib.fa_paged_workspace_size.restype = sz
        lib.fa_paged_attn.argtypes = ([vp] * 7 + [i, i, i, i, i, i, i64, i64, i64, vp, i64, i, vp]
                                      + [vp, i, i, i, i64, f, i, i, vp, sz, vp])
        lib.fa_paged_attn.restype = i
        lib.fa_fp8_workspace_size.argtypes = [i, i, i]
        lib.fa_fp8_workspace_size.restype = sz
        lib.fa_fp8_vt_stride.argtypes = [i]
        lib.fa_fp8_vt_stride.restype = i
        lib.fa_fp8_quantize.argtypes = [vp, vp, vp, vp, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, sz,
                                        vp]
        lib.fa_fp8_quantize.restype = i
        lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, vp]
        lib.fa_fwd_fp8.restype = i
        lib.fa_fp8_quantize_gqa.argtypes = [vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp, vp, vp, vp,
                                            vp, sz, vp]
        lib.fa_fp8_quantize_gqa.restype = i
        lib.fa_fwd_fp8_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, vp]
        lib.fa_fwd_fp8_gqa.restype = i
        lib.fa_dropout_p8.argtypes = [f]
        lib.fa_dropout_p8.restype = i
        lib.fa_debug_dropout_keep.argtypes = [vp, i, i, i, f, u64, u64, vp]
        lib.fa_debug_dropout_keep.restype = i
        lib.fa_debug_philox.argtypes = [vp, vp, i, ctypes.c_uint32, ctypes.c_uint32, vp]
        lib.fa_debug_philox.restype = i
        lib.fa_butterfly_mask.argtypes = [vp, i]
        lib.fa_butterfly_mask.restype = i
        lib.fa_device_status.argtypes = [vp, i]
        lib.fa_device_status.restype = i
        lib.fa_set_wait_timeout_ns.argtypes = [u64]
        lib.fa_set_wait_timeout_ns.restype = None
        lib.fa_test_inject_stall.argtypes = [i]
        lib.fa_test_inject_stall.restype = None
        lib.fa_status_string.argtypes = [i]
        lib.fa_status_string.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().fa_status_string(int(status)).decode()


def fa_status_string(status: int) -> str:
    return status_string(status)


def _stream(stream=None):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


_HERE = contextlib.nullcontext()


def _memory_on(stream, dev):
    """Context in which tensors are made for a call on `stream` of device `dev` (None: the current
    one). Memory that torch hands out is free in the order of the stream that is current then:
    work queued earlier on another one may still use it."""
    if stream is None:
        return _HERE
    if not isinstance(stream, torch.cuda.Stream):
        # (torch knows CUDA's handle 1, cudaStreamLegacy, as stream 0 only)
        handle = int(stream)
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle, device=dev)
    return torch.cuda.stream(stream)


def _given_out(stream, dev, *tensors):
    """Results made by _memory_on(stream, dev) will be used on the current stream too: once the
    caller drops them, their memory waits for the work queued there as well."""
    if stream is not None:
        here = torch.cuda.current_stream(dev)
        for t in tensors:
            t.record_stream(here)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(status: int, where: str):
    if status != FA_OK:
        raise FAError(status, where)


def _check_qkv(*ts):
    for t in ts:
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 4:
            raise ValueError("expected contiguous 4-D bf16 CUDA tensors [B, H, N, d]")


def _kv_heads(q, k, v) -> int:
    """K/V head count; q [B, H, N, d] with k, v [B, H_kv, N, d], H a multiple of H_kv."""
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, N, d) or tuple(v.shape) != tuple(k.shape) or H % Hkv != 0:
        raise ValueError("k and v must be [B, H_kv, N, d] with H a multiple of H_kv")
    return Hkv


def _opt_ptrs(block_mask, seqlens_k, B, N):
    """Pointers of the optional block mask (uint8 [nb, nb], nb = ceil(N / 128))
    and key lengths (int32 [B]). The kernels index both without bounds (the C
    entry points cannot know their sizes), so their shapes are checked here."""
    if block_mask is not None:
        nb = (int(N) + 127) // 128
        if (block_mask.dtype != torch.uint8 or not block_mask.is_cuda
                or not block_mask.is_contiguous() or tuple(block_mask.shape) != (nb, nb)):
            raise ValueError(f"block_mask must be a contiguous uint8 CUDA tensor [{nb}, {nb}]")
    if seqlens_k is not None:
        if (seqlens_k.dtype != torch.int32 or not seqlens_k.is_cuda
                or not seqlens_k.is_contiguous() or tuple(seqlens_k.shape) != (int(B),)):
            raise ValueError(f"seqlens_k must be a contiguous int32 CUDA tensor [{int(B)}]")
    return _ptr(block_mask), _ptr(seqlens_k)


# ----------------------------------------------------------------- C mirrors

def fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal=False, dropout_p=0.0, seed=0, offset=0,
           block_mask=None, seqlens_k=None, stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                         int(bool(causal)), float(dropout_p), int(seed), int(offset), bm, sl,
                         _stream(stream))


def fa_bwd_workspace_size(B, H, N, d) -> int:
    return int(load().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal=False, dropout_p=0.0,
           seed=0, offset=0, block_mask=None, seqlens_k=None, workspace=None, workspace_bytes=0,
           stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                         _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                         float(dropout_p), int(seed), int(offset), bm, sl, _ptr(workspace),
                         int(workspace_bytes), _stream(stream))


def fa_fwd_gqa(q, k, v, o, lse, B, H, H_kv, N, d, scale, causal=False, dropout_p=0.0, seed=0,
               offset=0, block_mask=None, seqlens_k=None, stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, H_kv, N, d,
                             float(scale), int(bool(causal)), float(dropout_p), int(seed),
                             int(offset), bm, sl, _stream(stream))


def fa_bwd_gqa(q, k, v, o, dout, lse, dq, dk, dv, B, H, H_kv, N, d, scale, causal=False,
               dropout_p=0.0, seed=0, offset=0, block_mask=None, seqlens_k=None, workspace=None,
               workspace_bytes=0, stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                             _ptr(dk), _ptr(dv), B, H, H_kv, N, d, float(scale),
                             int(bool(causal)), float(dropout_p), int(seed), int(offset), bm, sl,
                             _ptr(workspace), int(workspace_bytes), _stream(stream))


def fa_fwd_window(q, k, v, o, lse, B, H, H_kv, N, d, scale, causal=False, window_left=-1,
                  window_right=-1, dropout_p=0.0, seed=0, offset=0, block_mask=None,
                  seqlens_k=None, stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_fwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, H_kv, N, d,
                                float(scale), int(bool(causal)), int(window_left),
                                int(window_right), float(dropout_p), int(seed), int(offset), bm,
                                sl, _stream(stream))


def fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, B, H, H_kv, N, d, scale, causal=False,
                  window_left=-1, window_right=-1, dropout_p=0.0, seed=0, offset=0,
                  block_mask=None, seqlens_k=None, workspace=None, workspace_bytes=0,
                  stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_bwd_window(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, H, H_kv, N, d, float(scale),
                                int(bool(causal)), int(window_left), int(window_right),
                                float(dropout_p), int(seed), int(offset), bm, sl, _ptr(workspace),
                                int(workspace_bytes), _stream(stream))


def fa_bwd_preprocess(o, dout, B, H, N, d, workspace, workspace_bytes, stream=None) -> int:
    return load().fa_bwd_preprocess(_ptr(o), _ptr(dout), B, H, N, d, _ptr(workspace),
                                    int(workspace_bytes), _stream(stream))


def fa_bwd_dkdv(q, k, v, dout, lse, dk, dv, B, H, N, d, scale, causal=False, dropout_p=0.0,
                seed=0, offset=0, block_mask=None, seqlens_k=None, workspace=None,
                workspace_bytes=0, stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse), _ptr(dk),
                              _ptr(dv), B, H, N, d, float(scale), int(bool(causal)),
                              float(dropout_p), int(seed), int(offset), bm, sl, _ptr(workspace),
                              int(workspace_bytes), _stream(stream))


def fa_bwd_dq(q, k, v, dout, lse, dq, B, H, N, d, scale, causal=False, dropout_p=0.0, seed=0,
              offset=0, block_mask=None, seqlens_k=None, workspace=None, workspace_bytes=0,
              stream=None) -> int:
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(dout), _ptr(lse), _ptr(dq), B, H, N,
                            d, float(scale), int(bool(causal)), float(dropout_p), int(seed),
                            int(offset), bm, sl, _ptr(workspace), int(workspace_bytes),
                            _stream(stream))


def fa_bwd_noalloc(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal=False,
                   dropout_p=0.0, seed=0, offset=0, block_mask=None, seqlens_k=None,
                   stream=None) -> int:
    """fa_bwd for callers that cannot allocate device memory: the library uses
    its own static device scratch (B*H*N <= 2^22) instead of a workspace."""
    bm, sl = _opt_ptrs(block_mask, seqlens_k, B, N)
    return load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                 int(bool(causal)), float(dropout_p), int(seed), int(offset), bm,
                                 sl, _stream(stream))


def fa_decode_workspace_size(B, H, H_kv, Nq, Nk, d, num_ctas=0) -> int:
    return int(load().fa_decode_workspace_size(B, H, H_kv, Nq, Nk, d, num_ctas))


def fa_decode(q, k_cache, v_cache, o, lse, B, H, H_kv, Nq, Nk, d, scale, causal=False,
              seqlens_k=None, num_ctas=0, workspace=None, workspace_bytes=0, stream=None,
              window_left=-1) -> int:
    if seqlens_k is not None and (seqlens_k.dtype != torch.int32 or not seqlens_k.is_cuda
                                  or not seqlens_k.is_contiguous()
                                  or tuple(seqlens_k.shape) != (int(B),)):
        raise ValueError(f"seqlens_k must be a contiguous int32 CUDA tensor [{int(B)}]")
    return load().fa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse), B, H, H_kv,
                            Nq, Nk, d, float(scale), int(bool(causal)), int(window_left),
                            _ptr(seqlens_k), int(num_ctas), _ptr(workspace), int(workspace_bytes),
                            _stream(stream))


def fa_paged_write(k_new, v_new, k_pages, v_pages, k_scale, v_scale, type, num_pages, page_size,
                   H_kv, d, stride_page, stride_head, stride_row, page_table, table_stride,
                   max_pages, kv_lens, cu_seqlens_q, B, T, max_q, k_stride, v_stride,
                   stream=None) -> int:
    return load().fa_paged_write(_ptr(k_new), _ptr(v_new), _ptr(k_pages), _ptr(v_pages),
                                 _ptr(k_scale), _ptr(v_scale), type, num_pages, page_size, H_kv, d,
                                 stride_page, stride_head, stride_row, _ptr(page_table),
                                 table_stride, max_pages, _ptr(kv_lens), _ptr(cu_seqlens_q), B, T,
                                 max_q, k_stride, v_stride, _stream(stream))


def fa_paged_read(k_pages, v_pages, k_scale, v_scale, type, num_pages, page_size, H_kv, d,
                  stride_page, stride_head, stride_row, page_table, table_stride, max_pages,
                  kv_lens, B, N, k_out, v_out, stream=None) -> int:
    return load().fa_paged_read(_ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale), type,
                                num_pages, page_size, H_kv, d, stride_page, stride_head,
                                stride_row, _ptr(page_table), table_stride, max_pages,
                                _ptr(kv_lens), B, N, _ptr(k_out), _ptr(v_out), _stream(stream))


def fa_paged_workspace_size(H, H_kv, d, max_q, max_keys) -> int:
    return int(load().fa_paged_workspace_size(H, H_kv, d, max_q, max_keys))


def fa_paged_attn(q, k_pages, v_pages, k_scale, v_scale, o, lse, type, num_pages, page_size, H,
                  H_kv, d, stride_page, stride_head, stride_row, page_table, table_stride,
                  max_pages, kv_lens, cu_seqlens_q, B, T, max_q, q_stride, scale, causal=False,
                  window_left=-1, workspace=None, workspace_bytes=0, stream=None) -> int:
    return load().fa_paged_attn(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(k_scale),
                                _ptr(v_scale), _ptr(o), _ptr(lse), type, num_pages, page_size, H,
                                H_kv, d, stride_page, stride_head, stride_row, _ptr(page_table),
                                table_stride, max_pages, _ptr(kv_lens), _ptr(cu_seqlens_q), B, T,
                                max_q, q_stride, float(scale), int(bool(causal)),
                                int(window_left), _ptr(workspace), int(workspace_bytes),
                                _stream(stream))


def fa_fp8_workspace_size(B, H, d) -> int:
    return int(load().fa_fp8_workspace_size(B, H, d))


def fa_fp8_vt_stride(N) -> int:
    return int(load().fa_fp8_vt_stride(N))


def fa_fp8_quantize(q, k, v, signs, B, H, N, d, q8, k8, vt8, s_q, s_k, s_v, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().fa_fp8_quantize(_ptr(q), _ptr(k), _ptr(v), _ptr(signs), B, H, N, d, _ptr(q8),
                                  _ptr(k8), _ptr(vt8), _ptr(s_q), _ptr(s_k), _ptr(s_v),
                                  _ptr(workspace), int(workspace_bytes), _stream(stream))


def fa_fwd_fp8(q8, k8, vt8, s_q, s_k, s_v, o, lse, B, H, N, d, scale, causal=False,
               seqlens_k=None, stream=None) -> int:
    _, sl = _opt_ptrs(None, seqlens_k, B, N)
    return load().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(s_q), _ptr(s_k), _ptr(s_v),
                             _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(bool(causal)), sl,
                             _stream(stream))


def fa_fp8_quantize_gqa(q, k, v, signs, B, H, Hkv, N, d, q8, k8, vt8, s_q, s_k, s_v, workspace,
                        workspace_bytes, stream=None) -> int:
    return load().fa_fp8_quantize_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(signs), B, H, Hkv, N, d,
                                      _ptr(q8), _ptr(k8), _ptr(vt8), _ptr(s_q), _ptr(s_k),
                                      _ptr(s_v), _ptr(workspace), int(workspace_bytes),
                                      _stream(stream))


def fa_fwd_fp8_gqa(q8, k8, vt8, s_q, s_k, s_v, o, lse, B, H, Hkv, N, d, scale, causal=False,
                   seqlens_k=None, stream=None) -> int:
    _, sl = _opt_ptrs(None, seqlens_k, B, N)
    return load().fa_fwd_fp8_gqa(_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(s_q), _ptr(s_k), _ptr(s_v),
                                 _ptr(o), _ptr(lse), B, H, Hkv, N, d, float(scale),
                                 int(bool(causal)), sl, _stream(stream))


def fa_dropout_p8(p: float) -> int:
    return int(load().fa_dropout_p8(float(p)))


def fa_debug_dropout_keep(keep, B, H, N, dropout_p, seed=0, offset=0, stream=None) -> int:
    return load().fa_debug_dropout_keep(_ptr(keep), B, H, N, float(dropout_p), int(seed),
                                        int(offset), _stream(stream))


def fa_debug_philox(counters, out, n, key0, key1, stream=None) -> int:
    return load().fa_debug_philox(_ptr(counters), _ptr(out), int(n), int(key0), int(key1),
                                  _stream(stream))


def fa_butterfly_mask(nb: int) -> torch.Tensor:
    """Host uint8 [nb, nb] butterfly block mask from the library's generator."""
    m = torch.zeros((nb, nb), dtype=torch.uint8)
    _check(load().fa_butterfly_mask(ctypes.c_void_p(m.data_ptr()), nb), "fa_butterfly_mask")
    return m


def fa_device_status(stream=None, clear=True) -> int:
    return int(load().fa_device_status(_stream(stream), int(bool(clear))))


def fa_set_wait_timeout_ns(ns: int) -> None:
    load().fa_set_wait_timeout_ns(int(ns))


def fa_test_inject_stall(mode: int) -> None:
    load().fa_test_inject_stall(int(mode))


# ----------------------------------------------------------- conveniences

def fwd(q, k, v, scale=None, causal=False, dropout_p=0.0, seed=0, offset=0, block_mask=None,
        seqlens_k=None, stream=None, window=(-1, -1)):
    """Allocate O and lse with torch and run fa_fwd (fa_fwd_gqa when k and v
    have fewer heads than q, fa_fwd_window when window = (left, right) is
    set). Returns (o, lse)."""
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    Hkv = _kv_heads(q, k, v)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _memory_on(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if tuple(window) != (-1, -1):
        st = fa_fwd_window(q, k, v, o, lse, B, H, Hkv, N, d, scale, causal, window[0], window[1],
                           dropout_p, seed, offset, block_mask, seqlens_k, stream)
    elif Hkv == H:
        st = fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, dropout_p, seed, offset,
                    block_mask, seqlens_k, stream)
    else:
        st = fa_fwd_gqa(q, k, v, o, lse, B, H, Hkv, N, d, scale, causal, dropout_p, seed, offset,
                        block_mask, seqlens_k, stream)
    _check(st, "fa_fwd")
    _given_out(stream, q.device, o, lse)
    return o, lse


def bwd(q, k, v, o, dout, lse, scale=None, causal=False, dropout_p=0.0, seed=0, offset=0,
        block_mask=None, seqlens_k=None, workspace=None, stream=None, window=(-1, -1)):
    """Allocate dQ, dK, dV (and the workspace if not given) and run fa_bwd
    (fa_bwd_gqa when k and v have fewer heads than q, fa_bwd_window when
    window = (left, right) is set)."""
    _check_qkv(q, k, v, o, dout)
    B, H, N, d = q.shape
    Hkv = _kv_heads(q, k, v)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _memory_on(stream, q.device):
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        if workspace is None:
            workspace = torch.empty(fa_bwd_workspace_size(B, H, N, d), dtype=torch.uint8,
                                    device=q.device)
    if tuple(window) != (-1, -1):
        st = fa_bwd_window(q, k, v, o, dout, lse, dq, dk, dv, B, H, Hkv, N, d, scale, causal,
                           window[0], window[1], dropout_p, seed, offset, block_mask, seqlens_k,
                           workspace, workspace.numel(), stream)
    elif Hkv == H:
        st = fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, dropout_p, seed,
                    offset, block_mask, seqlens_k, workspace, workspace.numel(), stream)
    else:
        st = fa_bwd_gqa(q, k, v, o, dout, lse, dq, dk, dv, B, H, Hkv, N, d, scale, causal,
                        dropout_p, seed, offset, block_mask, seqlens_k, workspace,
                        workspace.numel(), stream)
    _check(st, "fa_bwd")
    _given_out(stream, q.device, dq, dk, dv)
    return dq, dk, dv


def decode(q, k_cache, v_cache, scale=None, causal=False, seqlens_k=None, num_ctas=0,
           stream=None, window_left=-1):
    """Allocate O, lse (and the workspace, if the split needs one) with torch and
    run fa_decode: q [B, H, Nq, d] over k_cache, v_cache [B, H_kv, Nk, d].
    Returns (o, lse)."""
    _check_qkv(q, k_cache, v_cache)
    B, H, Nq, d = q.shape
    _, Hkv, Nk, _ = k_cache.shape
    if tuple(v_cache.shape) != tuple(k_cache.shape) or k_cache.shape[0] != B or \
            k_cache.shape[3] != d:
        raise ValueError("k_cache and v_cache must be [B, H_kv, Nk, d] like q's B and d")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    ws_bytes = fa_decode_workspace_size(B, H, Hkv, Nq, Nk, d, num_ctas)
    with _memory_on(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device) if ws_bytes else None
    _check(fa_decode(q, k_cache, v_cache, o, lse, B, H, Hkv, Nq, Nk, d, scale, causal, seqlens_k,
                     num_ctas, ws, ws_bytes, stream, window_left), "fa_decode")
    _given_out(stream, q.device, o, lse)
    return o, lse


def fp8_quantize(q, k, v, signs=None, stream=None):
    """Allocate the e4m3 tensors and scales with torch and run fa_fp8_quantize
    (fa_fp8_quantize_gqa when k and v have fewer heads than q).
    Returns dict(q8, k8, vt8, s_q, s_k, s_v) (uint8 codes, fp32 scales)."""
    _check_qkv(q, k, v)
    Hkv = _kv_heads(q, k, v)
    B, H, N, d = q.shape
    dev = q.device
    Np = fa_fp8_vt_stride(N)
    wsb = fa_fp8_workspace_size(B, H, d)
    with _memory_on(stream, dev):
        out = dict(q8=torch.empty((B, H, N, d), dtype=torch.uint8, device=dev),
                   k8=torch.empty((B, Hkv, N, d), dtype=torch.uint8, device=dev),
                   vt8=torch.empty((B, Hkv, d, Np), dtype=torch.uint8, device=dev),
                   s_q=torch.empty((B, H), dtype=torch.float32, device=dev),
                   s_k=torch.empty((B, Hkv), dtype=torch.float32, device=dev),
                   s_v=torch.empty((B, Hkv, d), dtype=torch.float32, device=dev))
        ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    if Hkv == H:
        st = fa_fp8_quantize(q, k, v, signs, B, H, N, d, out["q8"], out["k8"], out["vt8"],
                             out["s_q"], out["s_k"], out["s_v"], ws, wsb, stream)
    else:
        st = fa_fp8_quantize_gqa(q, k, v, signs, B, H, Hkv, N, d, out["q8"], out["k8"],
                                 out["vt8"], out["s_q"], out["s_k"], out["s_v"], ws, wsb, stream)
    _check(st, "fa_fp8_quantize")
    _given_out(stream, dev, *out.values())
    return out


def fwd_fp8(qz, scale, causal=False, seqlens_k=None, stream=None):
    """Run fa_fwd_fp8 (fa_fwd_fp8_gqa with grouped K/V heads) on the output of
    fp8_quantize; returns (o bf16, lse)."""
    B, H, N, d = qz["q8"].shape
    Hkv = qz["k8"].shape[1]
    dev = qz["q8"].device
    with _memory_on(stream, dev):
        o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((B, H, N), dtype=torch.float32, device=dev)
    args = (qz["q8"], qz["k8"], qz["vt8"], qz["s_q"], qz["s_k"], qz["s_v"], o, lse)
    if Hkv == H:
        st = fa_fwd_fp8(*args, B, H, N, d, scale, causal, seqlens_k, stream)
    else:
        st = fa_fwd_fp8_gqa(*args, B, H, Hkv, N, d, scale, causal, seqlens_k, stream)
    _check(st, "fa_fwd_fp8")
    _given_out(stream, dev, o, lse)
    return o, lse


# ------------------------------------------------------------- paged caches

def paged_cache(num_pages, page_size, H_kv, d, e4m3=False, device="cuda"):
    """Allocate an empty paged cache: dict(k_pages, v_pages [num_pages, H_kv, page_size, d],
    bf16, or uint8 e4m3 codes with k_scale, v_scale uint8 [num_pages, H_kv, page_size];
    these are None for bf16). The keywords are those of paged_write, paged_read and
    paged_attn."""
    shape = (num_pages, H_kv, page_size, d)
    out = {}
    for n in ("k", "v"):
        out[n + "_pages"] = torch.empty(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16,
                                        device=device)
        out[n + "_scale"] = (torch.empty(shape[:3], dtype=torch.uint8, device=device) if e4m3
                             else None)
    return out


def _paged_batch(k_pages, v_pages, page_table, kv_lens, k_scale, v_scale):
    """Arguments that the paged calls share, checked: (cache type .. page_size), then (H_kv ..
    kv_lens), as the C entry points take them, B and the device's index."""
    shape, st, dtype = k_pages.shape, k_pages.stride(), k_pages.dtype
    if len(shape) != 4 or v_pages.shape != shape or v_pages.dtype != dtype:
        raise ValueError("k_pages and v_pages must be alike, [num_pages, H_kv, page_size, d]")
    P, Hkv, page, d = shape
    if v_pages.stride() != st or (st[3] != 1 and d > 1):
        raise ValueError("k_pages and v_pages must have the same strides, with d contiguous")
    dev = k_pages.get_device()
    if dev < 0 or v_pages.get_device() != dev:
        raise ValueError("k_pages and v_pages must be CUDA tensors on one device")
    if dtype == torch.bfloat16:
        kind = FA_CACHE_BF16
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bf16 cache has no scales")
    elif dtype in (torch.uint8, torch.float8_e4m3fn):
        kind = FA_CACHE_E4M3
        for t in (k_scale, v_scale):
            if (t is None or t.dtype != torch.uint8 or t.shape != shape[:3]
                    or not t.is_contiguous() or t.get_device() != dev):
                raise ValueError("an e4m3 cache needs k_scale and v_scale, contiguous uint8 "
                                 f"[{P}, {Hkv}, {page}], on the pages' device")
    else:
        raise ValueError("pages must be bf16, or e4m3 codes (uint8 or float8_e4m3fn)")
    table = page_table.shape
    if page_table.dtype != torch.int32 or len(table) != 2 or page_table.get_device() != dev:
        raise ValueError("page_table must be int32 [B, max_pages], on the pages' device")
    B, width = table
    if B < 1 or width < 1:
        raise ValueError("page_table must have a row and a page")
    ts, tc = page_table.stride()
    if tc != 1 and width > 1:
        raise ValueError("the rows of page_table must be contiguous")
    if (kv_lens.dtype != torch.int32 or kv_lens.shape != (B,) or kv_lens.get_device() != dev
            or not kv_lens.is_contiguous()):
        raise ValueError(f"kv_lens must be contiguous int32 [{B}], on the pages' device")
    # the stride of a dimension of size one is never used: any valid one stands for it
    sr = st[2] if page > 1 else d
    sh = st[1] if Hkv > 1 else sr * page
    sp = st[0] if P > 1 else sh * Hkv
    return ((kind, P, page), (Hkv, d, sp, sh, sr, page_table.data_ptr(),
                              ts if B > 1 else width, width, kv_lens.data_ptr()), B, dev)


def _new_rows(name, x, heads, d, dev):
    """Token stride of packed rows [T, heads, d] with heads and d contiguous."""
    shape = x.shape
    if (x.dtype != torch.bfloat16 or len(shape) != 3 or shape[1] != heads or shape[2] != d
            or x.get_device() != dev):
        raise ValueError(f"{name} must be bf16 [T, {heads}, {d}], on the pages' device")
    st, sh, sd = x.stride()
    if sd != 1 or (sh != d and heads > 1):
        raise ValueError(f"heads and d of {name} must be contiguous")
    return st if shape[0] > 1 else heads * d


def _offsets(cu, B, T, max_q, dev):
    """Pointer of cu_seqlens_q (checked) and max_q of a batch of T packed rows."""
    if cu is None:
        if T % B != 0 or (max_q is not None and max_q * B != T):
            raise ValueError("without cu_seqlens_q the rows must be B times max_q")
        return 0, T // B
    if (cu.dtype != torch.int32 or cu.shape != (B + 1,) or cu.get_device() != dev
            or not cu.is_contiguous()):
        raise ValueError(f"cu_seqlens_q must be contiguous int32 [{B + 1}], on the pages' device")
    return cu.data_ptr(), T if max_q is None else max_q


def _data(t):
    return 0 if t is None else t.data_ptr()


# The arguments of the paged entry points as their _block forms take them.
_WRITE_BLOCK = struct.Struct("=24q").pack
_READ_BLOCK = struct.Struct("=20q").pack
_ATTN_BLOCK = struct.Struct("=25qd4q").pack


def _call(name, dev, stream, block):
    """Call a C entry point, its arguments packed into `block`, on device `dev` and a stream of
    it (the current one if None)."""
    if stream is None:
        # the raw handle of the current stream, without a Stream object around it: a
        # decode step makes this call in microseconds
        handle = torch._C._cuda_getCurrentRawStream(dev)
    else:
        handle = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    f = getattr(load() if _lib is None else _lib, name)
    if torch._C._cuda_getDevice() == dev:
        status = f(block, handle)
    else:
        with torch.cuda.device(dev):
            status = f(block, handle)
    if status != FA_OK:
        raise FAError(status, name)


@functools.lru_cache(maxsize=4096)
def _paged_workspace_bytes(H, H_kv, d, max_q, max_keys, dev):
    with torch.cuda.device(dev):  # depends on the device's number of SMs
        return fa_paged_workspace_size(H, H_kv, d, max_q, max_keys)


def paged_write(k_new, v_new, k_pages, v_pages, page_table, kv_lens, cu_seqlens_q=None,
                k_scale=None, v_scale=None, stream=None):
    """Store new rows k_new, v_new [T, H_kv, d] into the pages (fa_paged_write). The new tokens
    of sequence b are rows cu_seqlens_q[b] .. cu_seqlens_q[b + 1] (T / B each without
    cu_seqlens_q) and take its last positions, kv_lens [B] counting them already."""
    head, batch, B, dev = _paged_batch(k_pages, v_pages, page_table, kv_lens, k_scale, v_scale)
    T = k_new.shape[0]
    ks = _new_rows("k_new", k_new, batch[0], batch[1], dev)
    vs = _new_rows("v_new", v_new, batch[0], batch[1], dev)
    if v_new.shape[0] != T:
        raise ValueError("k_new and v_new must have the same number of rows")
    cu, n = _offsets(cu_seqlens_q, B, T, None, dev)
    _call("fa_paged_write_block", dev, stream,
          _WRITE_BLOCK(k_new.data_ptr(), v_new.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                       _data(k_scale), _data(v_scale), *head, *batch, cu, B, T, n, ks, vs))


def paged_read(k_pages, v_pages, page_table, kv_lens, N, k_scale=None, v_scale=None, stream=None):
    """Copy positions 0 .. N - 1 of every sequence out of the pages (fa_paged_read): k and v,
    bf16 [B, H_kv, N, d], zeros behind each sequence. fwd and decode take them with
    seqlens_k=kv_lens."""
    head, batch, B, dev = _paged_batch(k_pages, v_pages, page_table, kv_lens, k_scale, v_scale)
    shape = (B, batch[0], N, batch[1])
    with _memory_on(stream, dev):
        k = k_pages.new_empty(shape, dtype=torch.bfloat16)
        v = k_pages.new_empty(shape, dtype=torch.bfloat16)
    _call("fa_paged_read_block", dev, stream,
          _READ_BLOCK(k_pages.data_ptr(), v_pages.data_ptr(), _data(k_scale), _data(v_scale),
                      *head, *batch, B, N, k.data_ptr(), v.data_ptr()))
    if stream is not None:
        _given_out(stream, dev, k, v)
    return k, v


def paged_attn(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens_q=None, max_q=None, scale=None,
               causal=False, window_left=-1, k_scale=None, v_scale=None, out=None, stream=None):
    """Attention of the new tokens q [T, H, d] over the cache (fa_paged_attn). The tokens of
    sequence b are rows cu_seqlens_q[b] .. cu_seqlens_q[b + 1] (T / B each without
    cu_seqlens_q); max_q bounds their number (T where it is not given: pass it, since up to 24
    rows H / H_kv * max_q run on a kernel of their own). Returns (o [T, H, d] bf16, lse [T, H] fp32); rows that
    belong to no sequence are not written. out = (o, lse) gives the buffers (not over q)."""
    head, batch, B, dev = _paged_batch(k_pages, v_pages, page_table, kv_lens, k_scale, v_scale)
    Hkv, d = batch[0], batch[1]
    if q.dim() != 3:
        raise ValueError("q must be [T, H, d]")
    T, H = q.shape[0], q.shape[1]
    qs = _new_rows("q", q, H, d, dev)
    cu, n = _offsets(cu_seqlens_q, B, T, max_q, dev)
    ws_bytes = _paged_workspace_bytes(H, Hkv, d, n, head[2] * batch[7], dev) if T > 0 else 0
    with _memory_on(stream, dev):
        if out is None:
            o = q.new_empty((T, H, d))
            lse = q.new_empty((T, H), dtype=torch.float32)
        ws = q.new_empty(ws_bytes, dtype=torch.uint8) if ws_bytes else None
    if out is not None:
        o, lse = out
        if (o.dtype != torch.bfloat16 or o.shape != (T, H, d) or not o.is_contiguous()
                or lse.dtype != torch.float32 or lse.shape != (T, H) or not lse.is_contiguous()
                or o.get_device() != dev or lse.get_device() != dev):
            raise ValueError(f"out must be contiguous: bf16 [{T}, {H}, {d}] and fp32 [{T}, {H}]")
        qp, op, lp = q.data_ptr(), o.data_ptr(), lse.data_ptr()
        q_end = qp + 2 * ((T - 1) * qs + H * d)
        if T > 0 and (qp < op + 2 * T * H * d and op < q_end or qp < lp + 4 * T * H and lp < q_end):
            raise ValueError("out may not overlap q: rows of q are read after others are written")
    if T == 0:
        return o, lse
    _call("fa_paged_attn_block", dev, stream,
          _ATTN_BLOCK(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _data(k_scale),
                      _data(v_scale), o.data_ptr(), lse.data_ptr(), *head, H, *batch, cu, B, T, n,
                      qs, 1.0 / math.sqrt(d) if scale is None else scale, bool(causal),
                      min(window_left, 0x7FFFFFFF), _data(ws), ws_bytes))
    if stream is not None and out is None:
        _given_out(stream, dev, o, lse)
    return o, lse

"""Thin ctypes binding of libspa.so (include/spa.h), with the same names.

Argument marshalling only: every step runs in the CUDA kernels behind the C-ABI.
PyTorch is used for device memory and the current stream. There is no CPU path:
importing this module without a built libspa.so raises, and every call needs CUDA
tensors.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

__all__ = ["SpaError", "lib", "spa_block_stats", "spa_select", "spa_sparse_attn_prefill",
           "spa_decode_workspace_bytes", "spa_sparse_attn_decode", "spa_get_device_error",
           "spa_status_string", "spa_last_error", "prefill", "decode", "LIB_PATH",
           "spa_prefill_host", "spa_prefill_host_workspace_bytes", "spa_selftest_wait_timeout",
           "spa_rope_frequencies", "spa_rope", "spa_rope_append", "spa_tree_workspace_bytes",
           "spa_sparse_attn_tree", "spa_attn_weight_workspace_bytes", "spa_attn_weight",
           "spa_evict_select", "spa_cache_gather", "decode_tree", "evict"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspa.so")

SPA_F32, SPA_BF16 = 0, 1
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_D = ctypes.c_double
_Z = ctypes.c_size_t

_lib = None


class SpaError(RuntimeError):
    """A libspa call returned a non-zero spa_status."""

    def __init__(self, fn: str, status: int, detail: str):
        self.status = status
        super().__init__(f"{fn}: {_status_name(status)} (status {status}): {detail}")


def lib() -> ctypes.CDLL:
    """The loaded libspa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libspa.so not found at {LIB_PATH}; build it with "
                              "`python -m block_sparse_long_stats_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.spa_block_stats.argtypes = [_P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P]
        L.spa_select.argtypes = [_P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _I, _I,
                                 _P, _I, _P, _P]
        L.spa_sparse_attn_prefill.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P,
                                              _F, _P, _P, _P]
        L.spa_decode_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
        L.spa_decode_workspace_bytes.restype = ctypes.c_size_t
        L.spa_sparse_attn_decode.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P,
                                             _F, _P, _P, _P]
        L.spa_rla_block_states.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P]
        L.spa_rla_prefill.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P,
                                      _P]
        L.spa_rla_decode_state.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P]
        L.spa_rla_decode_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I]
        L.spa_rla_decode_workspace_bytes.restype = ctypes.c_size_t
        L.spa_sparse_attn_decode_rla.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                                                 _I, _P, _F, _P, _P, _P, _P]
        L.spa_quantized_stats_bytes.argtypes = [_I, _I, _I, _I, _I]
        L.spa_quantized_stats_bytes.restype = ctypes.c_size_t
        L.spa_quantize_block_stats.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P]
        L.spa_block_stats_quantized.argtypes = [_P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I, _P]
        L.spa_select_quantized.argtypes = [_P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _I,
                                           _I, _P, _I, _P, _P]
        L.spa_select_score_order.argtypes = [_P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _I,
                                             _I, _I, _P, _I, _P, _P]
        L.spa_sparse_attn_prefill_early_stop.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                                         _P, _I, _P, _F, _I, _I, _F, _P, _P, _P,
                                                         _P]
        L.spa_pbs_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
        L.spa_pbs_workspace_bytes.restype = ctypes.c_size_t
        L.spa_pbs_permutation.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                          ctypes.c_size_t, _P, _P]
        L.spa_pbs_gather.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, _P]
        L.spa_select_segperm.argtypes = [_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                                         _F, _I, _I, _I, _P, _I, _P, _P]
        L.spa_sparse_attn_prefill_segperm.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                                      _I, _I, _P, _I, _P, _F, _P, _P, _P]
        L.spa_prefill_host_workspace_bytes.argtypes = [_I, _I, _I, _I, _I, _I, _I]
        L.spa_prefill_host_workspace_bytes.restype = ctypes.c_size_t
        L.spa_prefill_host.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _I,
                                       _I, _P, ctypes.c_size_t, _P]
        L.spa_rope_frequencies.argtypes = [_I, _D, _I, _D, _D, _D, _D, _P, ctypes.POINTER(_F)]
        L.spa_rope.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P,
                               _F, _P, _I, _I, _P]
        L.spa_rope_append.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                      _I, _I, _I, _P, _F, _P, _P, _I, _P]
        L.spa_tree_workspace_bytes.argtypes = [_I] * 7
        L.spa_tree_workspace_bytes.restype = _Z
        L.spa_sparse_attn_tree.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _I,
                                           _P, _F, _P, _Z, _P, _P, _P]
        L.spa_attn_weight_workspace_bytes.argtypes = [_I] * 5
        L.spa_attn_weight_workspace_bytes.restype = _Z
        L.spa_attn_weight.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _I, _P, _I, _P, _F, _P,
                                      _F, _P, _Z, _P, _P]
        L.spa_evict_select.argtypes = [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]
        L.spa_cache_gather.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _P, _I, _P, _P, _P, _P]
        L.spa_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.spa_selftest_wait_timeout.argtypes = [_I, _P]
        L.spa_status_string.argtypes = [_I]
        L.spa_status_string.restype = ctypes.c_char_p
        L.spa_last_error.restype = ctypes.c_char_p
        for f in ("spa_block_stats", "spa_select", "spa_sparse_attn_prefill",
                  "spa_sparse_attn_decode", "spa_get_device_error", "spa_rla_block_states",
                  "spa_rla_prefill", "spa_rla_decode_state", "spa_sparse_attn_decode_rla",
                  "spa_quantize_block_stats", "spa_select_quantized", "spa_select_score_order",
                  "spa_block_stats_quantized",
                  "spa_sparse_attn_prefill_early_stop", "spa_pbs_permutation", "spa_pbs_gather",
                  "spa_select_segperm", "spa_sparse_attn_prefill_segperm", "spa_prefill_host",
                  "spa_selftest_wait_timeout", "spa_rope_frequencies", "spa_rope",
                  "spa_rope_append", "spa_sparse_attn_tree", "spa_attn_weight", "spa_evict_select",
                  "spa_cache_gather"):
            getattr(L, f).restype = _I
        _lib = L
    return _lib


def _status_name(st: int) -> str:
    return lib().spa_status_string(st).decode()


def spa_status_string(status: int) -> str:
    return _status_name(status)


def spa_last_error() -> str:
    return lib().spa_last_error().decode()


def _check(fn: str, st: int):
    if st != 0:
        raise SpaError(fn, st, spa_last_error())


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libspa works on CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


_QFMT = {"int4": 0, "fp4": 1}


def _qfmt(fmt: str) -> int:
    if fmt not in _QFMT:
        raise ValueError(f"unknown record format {fmt!r} (int4 or fp4)")
    return _QFMT[fmt]


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SPA_BF16
    if t.dtype == torch.float32:
        return SPA_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def spa_block_stats(k: torch.Tensor, block: int, blk_begin: int = 0, blk_end: int | None = None,
                    mean: torch.Tensor | None = None, var: torch.Tensor | None = None,
                    stream=None):
    """Per-block key mean and variance: k [B,Hkv,T,d] -> mean, var [B,Hkv,nb,d] fp32."""
    B, Hkv, T, d = k.shape
    nb = -(-T // block)
    blk_end = nb if blk_end is None else blk_end
    if mean is None:
        mean = torch.empty((B, Hkv, nb, d), device=k.device, dtype=torch.float32)
    if var is None:
        var = torch.empty((B, Hkv, nb, d), device=k.device, dtype=torch.float32)
    _check("spa_block_stats", lib().spa_block_stats(_ptr(k), _dt(k), B, Hkv, T, d, block,
                                                    blk_begin, blk_end, _ptr(mean), _ptr(var),
                                                    _stream(stream)))
    return mean, var


def spa_select(q: torch.Tensor, mean: torch.Tensor, var: torch.Tensor, T: int, block: int,
               scale: float, top_p: float, n_sink: int = 1, n_local: int = 1, k_min: int = 0,
               idx: torch.Tensor | None = None, count: torch.Tensor | None = None,
               cap: int | None = None, stream=None):
    """Kept-block lists: q [B,Hq,Lq,d] (Lq = T or 1) -> idx [B,Hq,nq,cap], count [B,Hq,nq]."""
    B, Hq, Lq, d = q.shape
    Hkv = mean.shape[1]
    nb = -(-T // block)
    nq = -(-Lq // block)
    if idx is None:
        cap = nb if cap is None else cap
        idx = torch.empty((B, Hq, nq, cap), device=q.device, dtype=torch.int32)
    cap = idx.shape[-1]
    if count is None:
        count = torch.empty((B, Hq, nq), device=q.device, dtype=torch.int32)
    _check("spa_select", lib().spa_select(_ptr(q), _dt(q), _ptr(mean), _ptr(var), B, Hq, Hkv, Lq, T,
                                          d, block, scale, top_p, n_sink, n_local, k_min,
                                          _ptr(idx), cap, _ptr(count), _stream(stream)))
    return idx, count


def spa_quantized_stats_bytes(B: int, Hkv: int, T: int, d: int, block: int) -> int:
    return int(lib().spa_quantized_stats_bytes(B, Hkv, T, d, block))


def spa_quantize_block_stats(mean: torch.Tensor, var: torch.Tensor, T: int, block: int,
                             blk_begin: int = 0, blk_end: int | None = None,
                             qstats: torch.Tensor | None = None, fmt: str = "int4",
                             stream=None) -> torch.Tensor:
    """Microscale records [B, Hkv, nb, d + d/16] uint8 (fmt "int4" or "fp4") from fp32
    block statistics."""
    B, Hkv, nb, d = mean.shape
    if blk_end is None:
        blk_end = nb
    if qstats is None:
        qstats = torch.empty((B, Hkv, nb, d + d // 16), device=mean.device, dtype=torch.uint8)
    _check("spa_quantize_block_stats",
           lib().spa_quantize_block_stats(_ptr(mean), _ptr(var), B, Hkv, T, d, block, blk_begin,
                                          blk_end, _ptr(qstats), _qfmt(fmt), _stream(stream)))
    return qstats


def spa_block_stats_quantized(k: torch.Tensor, block: int, blk_begin: int, blk_end: int,
                              mean: torch.Tensor, var: torch.Tensor, qstats: torch.Tensor,
                              fmt: str = "int4", stream=None) -> None:
    """Statistics and records (fmt "int4" or "fp4") of blocks [blk_begin, blk_end) in
    one pass, into the caller's mean, var [B, Hkv, nb, d] and qstats [B, Hkv, nb,
    d + d/16]."""
    B, Hkv, T, d = k.shape
    _check("spa_block_stats_quantized",
           lib().spa_block_stats_quantized(_ptr(k), _dt(k), B, Hkv, T, d, block, blk_begin, blk_end,
                                           _ptr(mean), _ptr(var), _ptr(qstats), _qfmt(fmt),
                                           _stream(stream)))


def spa_select_quantized(q: torch.Tensor, qstats: torch.Tensor, T: int, block: int, scale: float,
                         top_p: float, n_sink: int = 1, n_local: int = 1, k_min: int = 0,
                         idx: torch.Tensor | None = None, count: torch.Tensor | None = None,
                         fmt: str = "int4", stream=None):
    """spa_select on quantised statistics (records in format fmt). Returns (idx, count)."""
    B, Hq, Lq, d = q.shape
    Hkv = qstats.shape[1]
    nb = -(-T // block)
    nq = -(-Lq // block)
    if idx is None:
        idx = torch.empty((B, Hq, nq, nb), device=q.device, dtype=torch.int32)
    if count is None:
        count = torch.empty((B, Hq, nq), device=q.device, dtype=torch.int32)
    _check("spa_select_quantized",
           lib().spa_select_quantized(_ptr(q), _dt(q), _ptr(qstats), _qfmt(fmt), B, Hq, Hkv, Lq,
                                      T, d, block, scale, top_p, n_sink, n_local, k_min, _ptr(idx),
                                      idx.shape[-1], _ptr(count), _stream(stream)))
    return idx, count


def spa_select_score_order(q: torch.Tensor, mean: torch.Tensor, var: torch.Tensor, block: int,
                           scale: float, top_p: float, n_sink: int = 1, n_local: int = 1,
                           k_min: int = 0, idx: torch.Tensor | None = None,
                           count: torch.Tensor | None = None, stream=None):
    """Prefill selection with the kept lists in traversal order. Returns (idx, count)."""
    B, Hq, L, d = q.shape
    Hkv = mean.shape[1]
    nb = -(-L // block)
    if idx is None:
        idx = torch.empty((B, Hq, nb, nb), device=q.device, dtype=torch.int32)
    if count is None:
        count = torch.empty((B, Hq, nb), device=q.device, dtype=torch.int32)
    _check("spa_select_score_order",
           lib().spa_select_score_order(_ptr(q), _dt(q), _ptr(mean), _ptr(var), B, Hq, Hkv, L, d,
                                        block, scale, top_p, n_sink, n_local, k_min, _ptr(idx),
                                        idx.shape[-1], _ptr(count), _stream(stream)))
    return idx, count


def spa_sparse_attn_prefill_early_stop(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                       block: int, idx: torch.Tensor, count: torch.Tensor,
                                       scale: float, tau: float, n_sink: int = 1, n_local: int = 1,
                                       out: torch.Tensor | None = None,
                                       lse: torch.Tensor | None = None, want_lse: bool = False,
                                       processed: torch.Tensor | None = None, stream=None):
    """Attention over the prefix of score-ordered lists kept by the early stop.
    Returns (out, lse or None, processed [B, Hq, nq] int32)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, L), device=q.device, dtype=torch.float32)
    if processed is None:
        processed = torch.empty(count.shape, device=q.device, dtype=torch.int32)
    _check("spa_sparse_attn_prefill_early_stop",
           lib().spa_sparse_attn_prefill_early_stop(_ptr(q), _ptr(k), _ptr(v), _dt(q), B, Hq, Hkv,
                                                    L, d, block, _ptr(idx), idx.shape[-1],
                                                    _ptr(count), scale, n_sink, n_local, tau,
                                                    _ptr(out), _ptr(lse), _ptr(processed),
                                                    _stream(stream)))
    return out, lse, processed


def _hptr(t: torch.Tensor):
    if t.is_cuda:
        raise ValueError("spa_prefill_host takes host (CPU) tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def spa_prefill_host_workspace_bytes(dtype: torch.dtype, B: int, Hq: int, Hkv: int, L: int,
                                     d: int, block: int) -> int:
    """Device workspace bytes spa_prefill_host needs for these sizes."""
    dt = SPA_BF16 if dtype == torch.bfloat16 else SPA_F32
    return int(lib().spa_prefill_host_workspace_bytes(dt, B, Hq, Hkv, L, d, block))


def spa_prefill_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block: int,
                     top_p: float, scale: float | None = None, n_sink: int = 1, n_local: int = 1,
                     k_min: int = 0, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The whole prefill path from host tensors (pinned for copy/compute overlap):
    q [B,Hq,L,d], k, v [B,Hkv,L,d] on the CPU -> out [B,Hq,L,d] on the CPU. Asynchronous
    on `stream`: synchronise it before reading out."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=q.is_pinned())
    need = spa_prefill_host_workspace_bytes(q.dtype, B, Hq, Hkv, L, d, block)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    _check("spa_prefill_host",
           lib().spa_prefill_host(_hptr(q), _hptr(k), _hptr(v), _hptr(out), _dt(q), B, Hq, Hkv, L,
                                  d, block, scale, top_p, n_sink, n_local, k_min, _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def spa_pbs_workspace_bytes(B: int, Hq: int, Hkv: int, L: int, block: int) -> int:
    return int(lib().spa_pbs_workspace_bytes(B, Hq, Hkv, L, block))


def spa_pbs_permutation(q: torch.Tensor, k: torch.Tensor, block: int, seg_blocks: int,
                        scale: float, perm: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Segmented key permutation: perm [B, Hkv, L] int32 (original index per position)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if perm is None:
        perm = torch.empty((B, Hkv, L), device=q.device, dtype=torch.int32)
    need = spa_pbs_workspace_bytes(B, Hq, Hkv, L, block)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check("spa_pbs_permutation",
           lib().spa_pbs_permutation(_ptr(q), _ptr(k), _dt(q), B, Hq, Hkv, L, d, block, seg_blocks,
                                     scale, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _ptr(perm),
                                     _stream(stream)))
    return perm


def spa_pbs_gather(x: torch.Tensor, perm: torch.Tensor, xp: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The permuted copy of K or V: xp[b, g, p] = x[b, g, perm[b, g, p]]."""
    B, Hkv, L, d = x.shape
    if xp is None:
        xp = torch.empty_like(x)
    _check("spa_pbs_gather",
           lib().spa_pbs_gather(_ptr(x), _dt(x), B, Hkv, L, d, _ptr(perm), _ptr(xp),
                                _stream(stream)))
    return xp


def spa_select_segperm(q: torch.Tensor, mean: torch.Tensor, var: torch.Tensor,
                       mean_p: torch.Tensor, var_p: torch.Tensor, block: int, seg_blocks: int,
                       scale: float, top_p: float, n_sink: int = 1, n_local: int = 1,
                       k_min: int = 0, idx: torch.Tensor | None = None,
                       count: torch.Tensor | None = None, stream=None):
    """Prefill selection on the segment-permuted layout. Returns (idx, count)."""
    B, Hq, L, d = q.shape
    Hkv = mean.shape[1]
    nb = -(-L // block)
    if idx is None:
        idx = torch.empty((B, Hq, nb, nb), device=q.device, dtype=torch.int32)
    if count is None:
        count = torch.empty((B, Hq, nb), device=q.device, dtype=torch.int32)
    _check("spa_select_segperm",
           lib().spa_select_segperm(_ptr(q), _dt(q), _ptr(mean), _ptr(var), _ptr(mean_p),
                                    _ptr(var_p), B, Hq, Hkv, L, d, block, seg_blocks, scale, top_p,
                                    n_sink, n_local, k_min, _ptr(idx), idx.shape[-1], _ptr(count),
                                    _stream(stream)))
    return idx, count


def spa_sparse_attn_prefill_segperm(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                    kp: torch.Tensor, vp: torch.Tensor, block: int, seg_blocks: int,
                                    idx: torch.Tensor, count: torch.Tensor, scale: float,
                                    out: torch.Tensor | None = None,
                                    lse: torch.Tensor | None = None, want_lse: bool = False,
                                    stream=None):
    """Block-sparse prefill on the segment-permuted layout. Returns (out, lse or None)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, L), device=q.device, dtype=torch.float32)
    _check("spa_sparse_attn_prefill_segperm",
           lib().spa_sparse_attn_prefill_segperm(_ptr(q), _ptr(k), _ptr(v), _ptr(kp), _ptr(vp),
                                                 _dt(q), B, Hq, Hkv, L, d, block, seg_blocks,
                                                 _ptr(idx), idx.shape[-1], _ptr(count), scale,
                                                 _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


def spa_sparse_attn_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block: int,
                            idx: torch.Tensor, count: torch.Tensor, scale: float,
                            out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            want_lse: bool = False, stream=None):
    """Block-sparse causal attention over the kept blocks. Returns (out, lse or None)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, L), device=q.device, dtype=torch.float32)
    _check("spa_sparse_attn_prefill",
           lib().spa_sparse_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _dt(q), B, Hq, Hkv, L, d,
                                         block, _ptr(idx), idx.shape[-1], _ptr(count), scale,
                                         _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


def spa_rla_block_states(k: torch.Tensor, v: torch.Tensor, block: int, blk_begin: int = 0,
                         blk_end: int | None = None, states: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Per-block linear-attention states W_j[e][c] = sum_u v_u[e] exp(k_u[c]):
    [B, Hkv, nb, d, d] bf16."""
    B, Hkv, T, d = k.shape
    nb = -(-T // block)
    if blk_end is None:
        blk_end = nb
    if states is None:
        states = torch.empty((B, Hkv, nb, d, d), device=k.device, dtype=torch.bfloat16)
    _check("spa_rla_block_states",
           lib().spa_rla_block_states(_ptr(k), _ptr(v), _dt(k), B, Hkv, T, d, block, blk_begin,
                                      blk_end, _ptr(states), _stream(stream)))
    return states


def spa_rla_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, states: torch.Tensor,
                    block: int, idx: torch.Tensor, count: torch.Tensor,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Residual Linear Attention branch of prefill: [B, Hq, L, d] fp32."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    if out is None:
        out = torch.empty((B, Hq, L, d), device=q.device, dtype=torch.float32)
    _check("spa_rla_prefill",
           lib().spa_rla_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(states), _dt(q), B, Hq, Hkv, L, d,
                                 block, _ptr(idx), idx.shape[-1], _ptr(count), _ptr(out),
                                 _stream(stream)))
    return out


def spa_rla_decode_state(kc: torch.Tensor, vc: torch.Tensor, tok_begin: int = 0,
                         tok_end: int | None = None, state: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Adds sum_{t in [tok_begin, tok_end)} v_t exp(k_t)^T into state [B, Hkv, d, d]
    fp32 (a zeroed state is made when none is given)."""
    B, Hkv, T, d = kc.shape
    if tok_end is None:
        tok_end = T
    if state is None:
        state = torch.zeros((B, Hkv, d, d), device=kc.device, dtype=torch.float32)
    _check("spa_rla_decode_state",
           lib().spa_rla_decode_state(_ptr(kc), _ptr(vc), _dt(kc), B, Hkv, T, d, tok_begin,
                                      tok_end, _ptr(state), _stream(stream)))
    return state


def spa_rla_decode_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, d: int, block: int) -> int:
    return int(lib().spa_rla_decode_workspace_bytes(B, Hq, Hkv, T, d, block))


def spa_sparse_attn_decode_rla(q: torch.Tensor, kc: torch.Tensor, vc: torch.Tensor,
                               state: torch.Tensor, block: int, idx: torch.Tensor,
                               count: torch.Tensor, scale: float,
                               workspace: torch.Tensor | None = None,
                               out: torch.Tensor | None = None,
                               out_rla: torch.Tensor | None = None, stream=None):
    """Decode attention plus the linear branch over the unkept blocks.
    Returns (out [B,Hq,1,d] bf16, out_rla [B,Hq,1,d] fp32)."""
    B, Hq, _, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    if workspace is None:
        n = spa_rla_decode_workspace_bytes(B, Hq, Hkv, T, d, block)
        workspace = torch.empty((max(n, 16),), device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if out_rla is None:
        out_rla = torch.empty(q.shape, device=q.device, dtype=torch.float32)
    _check("spa_sparse_attn_decode_rla",
           lib().spa_sparse_attn_decode_rla(_ptr(q), _ptr(kc), _ptr(vc), _ptr(state), _dt(q), B,
                                            Hq, Hkv, T, d, block, _ptr(idx), idx.shape[-1],
                                            _ptr(count), scale, _ptr(workspace), _ptr(out),
                                            _ptr(out_rla), _stream(stream)))
    return out, out_rla


def spa_decode_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, d: int, block: int) -> int:
    return int(lib().spa_decode_workspace_bytes(B, Hq, Hkv, T, d, block))


def spa_sparse_attn_decode(q: torch.Tensor, kc: torch.Tensor, vc: torch.Tensor, block: int,
                           idx: torch.Tensor, count: torch.Tensor, scale: float,
                           workspace: torch.Tensor | None = None,
                           out: torch.Tensor | None = None, stream=None):
    """Decode attention for one query per sequence: q [B,Hq,1,d] -> out [B,Hq,1,d]."""
    B, Hq, _, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    if workspace is None:
        n = spa_decode_workspace_bytes(B, Hq, Hkv, T, d, block)
        workspace = torch.empty((max(n, 16),), device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    _check("spa_sparse_attn_decode",
           lib().spa_sparse_attn_decode(_ptr(q), _ptr(kc), _ptr(vc), _dt(q), B, Hq, Hkv, T, d,
                                        block, _ptr(idx), idx.shape[-1], _ptr(count), scale,
                                        _ptr(workspace), _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------- serving operators

_ROPE_LAYOUT = {"half": 0, "interleaved": 1}
_ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("l", ctypes.c_int64)]


class _On:
    """The device of `t` current, and `stream` (if given) too, so that outputs and
    workspaces are allocated where they are used; yields the raw stream."""

    def __init__(self, t: torch.Tensor, stream):
        self.dev, self.stream, self.ctx = t.device, stream, None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device != self.dev:
                raise ValueError("the stream is on another device than the tensors")
            self.ctx = torch.cuda.stream(self.stream)
        elif torch.cuda.current_device() != self.dev.index:
            self.ctx = torch.cuda.device(self.dev)
        if self.ctx is not None:
            self.ctx.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _enqueue(call, t: torch.Tensor, stream):
    """call(raw stream) on the tensor's device and on `stream`, or the current one."""
    if not t.is_cuda:
        raise ValueError("libspa works on CUDA tensors only")
    dev = t.get_device()
    if stream is None and dev == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(dev))
    with _On(t, stream) as st:
        return call(st)


def _mismatch(t, name, shape, dtype, dev):
    return ValueError(f"{name} must be {tuple(shape)} {dtype} on cuda:{dev}, "
                      f"got {tuple(t.shape)} {t.dtype} on {t.device}")


def _arg(t: torch.Tensor | None, name: str, shape, dtype, dev: int) -> int | None:
    """The address of a dense tensor of exactly this shape, type and device."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != dev or t.shape != shape:
        raise _mismatch(t, name, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _strided(t: torch.Tensor, name: str, shape, dtype, dev: int):
    """(address, strides or None where dense) of a [B, H, L, d] view with dense rows."""
    if t.dtype != dtype or t.get_device() != dev or t.shape != shape:
        raise _mismatch(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t.data_ptr(), None
    sb, sh, sl, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"the features of {name} must be contiguous")
    return t.data_ptr(), ctypes.byref(_Strides(sb, sh, sl))


def _layout(layout: str) -> int:
    if layout not in _ROPE_LAYOUT:
        raise ValueError(f"unknown rotary layout {layout!r} (half or interleaved)")
    return _ROPE_LAYOUT[layout]


def _rope_freqs(freqs: torch.Tensor) -> int:
    if freqs.dtype != torch.float64 or freqs.is_cuda or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a one-dimensional float64 tensor on the CPU")
    return freqs.data_ptr()


def spa_rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none",
                         factor: float = 1.0, trained: float = 0.0, fast: float = 32.0,
                         slow: float = 1.0):
    """Frequencies (float64 [rot/2], CPU) and the factor on the rotated values, for
    scaling "none", "linear", "ntk" or "parts"."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"unknown scaling {scaling!r} (none, linear, ntk or parts)")
    freqs = torch.empty(max(rot // 2, 0), dtype=torch.float64)
    m = ctypes.c_float(1.0)
    _check("spa_rope_frequencies",
           lib().spa_rope_frequencies(rot, base, _ROPE_SCALING[scaling], factor, trained, fast, slow,
                                      freqs.data_ptr() or None, ctypes.byref(m)))
    return freqs, m.value


def spa_rope(q: torch.Tensor, k: torch.Tensor | None, freqs: torch.Tensor, mscale: float = 1.0,
             layout: str = "half", pos: torch.Tensor | None = None, pos0: int = 0,
             backward: bool = False, q_out: torch.Tensor | None = None,
             k_out: torch.Tensor | None = None, stream=None):
    """Rotates q [B,Hq,L,d] and k [B,Hkv,L,d] (or None) of any strides with dense rows:
    -> (q_out, k_out or None), dense unless given. backward: the transposed rotation."""
    B, Hq, L, d = q.shape
    dev, dt = q.get_device(), q.dtype

    def call(st):
        nonlocal q_out, k_out
        qp, qs = _strided(q, "q", q.shape, dt, dev)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            qop, qos = q_out.data_ptr(), None
        else:
            qop, qos = _strided(q_out, "q_out", q.shape, dt, dev)
        kp = ks = kop = kos = None
        Hkv = 0
        if k is not None:
            Hkv = k.shape[1]
            shape = (B, Hkv, L, d)
            kp, ks = _strided(k, "k", shape, dt, dev)
            if k_out is None:
                k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
                kop, kos = k_out.data_ptr(), None
            else:
                kop, kos = _strided(k_out, "k_out", shape, dt, dev)
        elif k_out is not None:
            raise ValueError("k_out without k")
        _check("spa_rope",
               lib().spa_rope(qp, qs, qop, qos, kp, ks, kop, kos, _dt(q), B, Hq, Hkv, L, d,
                              2 * freqs.numel(), _layout(layout), _rope_freqs(freqs), mscale,
                              _arg(pos, "pos", (B, L), torch.int32, dev), pos0, int(backward), st))
        return q_out, k_out

    return _enqueue(call, q, stream)


def spa_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kc: torch.Tensor,
                    vc: torch.Tensor, freqs: torch.Tensor, mscale: float = 1.0,
                    rows: torch.Tensor | None = None, row0: int = 0, layout: str = "half",
                    pos: torch.Tensor | None = None, q_out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Rotates a step's new q (-> q_out) and k, and writes the rotated k and v into rows
    rows[b] + t (or row0 + t) of the caches kc, vc [B,Hkv,T,d]."""
    B, Hq, L, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    dev, dt = q.get_device(), q.dtype

    def call(st):
        nonlocal q_out
        qp, qs = _strided(q, "q", q.shape, dt, dev)
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            qop, qos = q_out.data_ptr(), None
        else:
            qop, qos = _strided(q_out, "q_out", q.shape, dt, dev)
        kp, ks = _strided(k, "k", (B, Hkv, L, d), dt, dev)
        vp, vs = _strided(v, "v", (B, Hkv, L, d), dt, dev)
        _check("spa_rope_append",
               lib().spa_rope_append(qp, qs, qop, qos, kp, ks, vp, vs,
                                     _arg(kc, "kc", (B, Hkv, T, d), dt, dev),
                                     _arg(vc, "vc", (B, Hkv, T, d), dt, dev), _dt(q), B, Hq, Hkv, L,
                                     T, d, 2 * freqs.numel(), _layout(layout), _rope_freqs(freqs),
                                     mscale, _arg(pos, "pos", (B, L), torch.int32, dev),
                                     _arg(rows, "rows", (B,), torch.int32, dev), row0, st))
        return q_out

    return _enqueue(call, q, stream)


def _lists(idx, count, B, Hq, nq, dev):
    """(address, cap, address) of kept lists, or of none."""
    if idx is None and count is None:
        return None, 0, None
    if idx is None or count is None:
        raise ValueError("idx and count go together")
    if idx.dim() != 4:
        raise ValueError("idx must be [B, Hq, nq, cap]")
    cap = idx.shape[3]
    return (_arg(idx, "idx", (B, Hq, nq, cap), torch.int32, dev), cap,
            _arg(count, "count", (B, Hq, nq), torch.int32, dev))


@functools.lru_cache(maxsize=256)
def spa_tree_workspace_bytes(B: int, Hq: int, Hkv: int, n: int, T: int, d: int, block: int) -> int:
    return int(lib().spa_tree_workspace_bytes(B, Hq, Hkv, n, T, d, block))


def spa_sparse_attn_tree(q: torch.Tensor, kc: torch.Tensor, vc: torch.Tensor,
                         parents: torch.Tensor, block: int, idx: torch.Tensor | None,
                         count: torch.Tensor | None, scale: float,
                         lens: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         want_lse: bool = False, stream=None):
    """Attention of a tree of n drafted tokens, q [B,Hq,n,d], that sit in the caches
    [B,Hkv,T,d] behind lens[b] tokens (T - n without lens); parents [B,n] int32, lists as
    for decode or None. Returns (out, lse or None)."""
    B, Hq, n, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    dev, dt = q.get_device(), q.dtype

    def call(st):
        nonlocal workspace, out, lse
        need = spa_tree_workspace_bytes(B, Hq, Hkv, n, T, d, block)
        if workspace is None:
            workspace = q.new_empty((max(need, 16),), dtype=torch.uint8)
        elif not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError("the workspace must be contiguous and on the tensors' device")
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
            op = out.data_ptr()
        else:
            op = _arg(out, "out", q.shape, dt, dev)
        if lse is None and want_lse:
            lse = q.new_empty((B, Hq, n), dtype=torch.float32)
            lp = lse.data_ptr()
        else:
            lp = _arg(lse, "lse", (B, Hq, n), torch.float32, dev)
        ip, cap, cp = _lists(idx, count, B, Hq, 1, dev)
        _check("spa_sparse_attn_tree",
               lib().spa_sparse_attn_tree(_arg(q, "q", q.shape, dt, dev),
                                          _arg(kc, "kc", (B, Hkv, T, d), dt, dev),
                                          _arg(vc, "vc", (B, Hkv, T, d), dt, dev), _dt(q), B, Hq, Hkv,
                                          n, T, d, block, _arg(parents, "parents", (B, n), torch.int32, dev),
                                          _arg(lens, "lens", (B,), torch.int32, dev), ip, cap, cp,
                                          scale, workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(),
                                          op, lp, st))
        return out, lse

    return _enqueue(call, q, stream)


@functools.lru_cache(maxsize=256)
def spa_attn_weight_workspace_bytes(B: int, Hkv: int, Lq: int, T: int, block: int) -> int:
    return int(lib().spa_attn_weight_workspace_bytes(B, Hkv, Lq, T, block))


def spa_attn_weight(q: torch.Tensor, k: torch.Tensor, lse: torch.Tensor, scale: float,
                    block: int = 128, idx: torch.Tensor | None = None,
                    count: torch.Tensor | None = None, lens: torch.Tensor | None = None,
                    prev: torch.Tensor | None = None, decay: float = 1.0,
                    workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Attention weight that the sequence's last Lq queries, q [B,Hq,Lq,d] with their lse
    [B,Hq,Lq], give every key of k [B,Hkv,T,d], added to decay * prev: [B,Hkv,T] fp32. The
    lse has to be over the keys that a query sees here: prefill's, or that of a tree's root
    or chain (of a tree with branches: of the accepted path, its rows copied together)."""
    B, Hq, Lq, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    dev, dt = q.get_device(), q.dtype

    def call(st):
        nonlocal workspace, out
        ip, cap, cp = None, 0, None
        if idx is not None or count is not None:
            nq = (T - 1) // block - (T - Lq) // block + 1 if block > 0 else 0
            ip, cap, cp = _lists(idx, count, B, Hq, nq, dev)
        if workspace is None:
            need = spa_attn_weight_workspace_bytes(B, Hkv, Lq, T, 0 if idx is None else block)
            workspace = q.new_empty((max(need, 16),), dtype=torch.uint8)
        elif not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError("the workspace must be contiguous and on the tensors' device")
        if out is None:
            out = q.new_empty((B, Hkv, T), dtype=torch.float32)
            op = out.data_ptr()
        else:
            op = _arg(out, "out", (B, Hkv, T), torch.float32, dev)
        _check("spa_attn_weight",
               lib().spa_attn_weight(_arg(q, "q", q.shape, dt, dev), _arg(k, "k", (B, Hkv, T, d), dt, dev),
                                     _dt(q), B, Hq, Hkv, Lq, T, d,
                                     _arg(lse, "lse", (B, Hq, Lq), torch.float32, dev),
                                     _arg(lens, "lens", (B,), torch.int32, dev), block, ip, cap, cp, scale,
                                     _arg(prev, "prev", (B, Hkv, T), torch.float32, dev), decay,
                                     workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     op, st))
        return out

    return _enqueue(call, q, stream)


def spa_evict_select(score: torch.Tensor, n_keep: int, n_sink: int = 4, n_recent: int = 0,
                     lens: torch.Tensor | None = None, keep: torch.Tensor | None = None,
                     count: torch.Tensor | None = None, stream=None):
    """The n_keep keys of score [B,Hkv,T] fp32 that stay: ascending keep [B,Hkv,n_keep] int32
    (-1 behind the last) and count [B] int32."""
    B, Hkv, T = score.shape
    dev = score.get_device()

    def call(st):
        nonlocal keep, count
        if keep is None:
            keep = score.new_empty((B, Hkv, max(n_keep, 0)), dtype=torch.int32)
        if count is None:
            count = score.new_empty((B,), dtype=torch.int32)
        _check("spa_evict_select",
               lib().spa_evict_select(_arg(score, "score", (B, Hkv, T), torch.float32, dev),
                                      _arg(lens, "lens", (B,), torch.int32, dev), B, Hkv, T, n_keep, n_sink,
                                      n_recent, _arg(keep, "keep", (B, Hkv, n_keep), torch.int32, dev),
                                      _arg(count, "count", (B,), torch.int32, dev), st))
        return keep, count

    return _enqueue(call, score, stream)


def spa_cache_gather(kc: torch.Tensor, vc: torch.Tensor, keep: torch.Tensor,
                     count: torch.Tensor | None = None, score: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                     score_out: torch.Tensor | None = None, stream=None):
    """The rows of kc, vc [B,Hkv,T,d] (and of score) that keep [B,Hkv,n_keep] names, closed up
    in k_out, v_out [B,Hkv,T_out,d] (T_out >= n_keep; new ones of n_keep rows, or of k_out's,
    zero behind the last, where none are given). Returns (k_out, v_out, score_out or None)."""
    B, Hkv, T, d = kc.shape
    n_keep = keep.shape[2]
    dev, dt = kc.get_device(), kc.dtype

    def call(st):
        nonlocal k_out, v_out, score_out
        T_out = n_keep if k_out is None else k_out.shape[2]
        new = kc.new_empty if count is None and T_out == n_keep else kc.new_zeros
        if k_out is None:
            k_out = new((B, Hkv, T_out, d))
        if v_out is None:
            v_out = new((B, Hkv, T_out, d))
        if score_out is None and score is not None:
            score_out = new((B, Hkv, T_out), dtype=torch.float32)
        _check("spa_cache_gather",
               lib().spa_cache_gather(_arg(kc, "kc", (B, Hkv, T, d), dt, dev),
                                      _arg(vc, "vc", (B, Hkv, T, d), dt, dev),
                                      _arg(score, "score", (B, Hkv, T), torch.float32, dev), _dt(kc), B, Hkv,
                                      T, d, _arg(keep, "keep", (B, Hkv, n_keep), torch.int32, dev), n_keep,
                                      _arg(count, "count", (B,), torch.int32, dev), T_out,
                                      _arg(k_out, "k_out", (B, Hkv, T_out, d), dt, dev),
                                      _arg(v_out, "v_out", (B, Hkv, T_out, d), dt, dev),
                                      _arg(score_out, "score_out", (B, Hkv, T_out), torch.float32, dev), st))
        return k_out, v_out, score_out

    return _enqueue(call, kc, stream)


def spa_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Enqueues the bounded-wait self-test: a wait that nothing completes runs out
    after limit_us and records SPA_DEVERR_TIMEOUT (read it with spa_get_device_error)."""
    _check("spa_selftest_wait_timeout", lib().spa_selftest_wait_timeout(limit_us, _stream(stream)))


def spa_get_device_error() -> int:
    """Reads and clears the device error word (synchronises); 0 means no error."""
    code = ctypes.c_int(0)
    st = lib().spa_get_device_error(ctypes.byref(code))
    if st not in (0, 4):
        _check("spa_get_device_error", st)
    return code.value


def prefill(q, k, v, block: int, top_p: float, scale: float | None = None, n_sink: int = 1,
            n_local: int = 1, k_min: int = 0, want_lse: bool = False, stream=None, rope=None,
            rope_layout: str = "half"):
    """The whole prefill path: (rotary positions) -> block stats -> selection -> sparse
    attention.

    rope: None, or the (freqs, mscale) of spa_rope_frequencies for q and k that are not
    rotated yet (of any strides with dense rows).
    Returns dict(out, lse, idx, count, mean, var), with rope also the rotated q and k.
    """
    T = k.shape[2]
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    rotated = {}
    if rope is not None:
        q, k = spa_rope(q, k, *rope, layout=rope_layout, stream=stream)
        rotated = {"q": q, "k": k}
    mean, var = spa_block_stats(k, block, stream=stream)
    idx, count = spa_select(q, mean, var, T, block, scale, top_p, n_sink, n_local, k_min,
                            stream=stream)
    out, lse = spa_sparse_attn_prefill(q, k, v, block, idx, count, scale, want_lse=want_lse,
                                       stream=stream)
    return {"out": out, "lse": lse, "idx": idx, "count": count, "mean": mean, "var": var, **rotated}


def decode(q, kc, vc, block: int, top_p: float, mean=None, var=None, scale: float | None = None,
           n_sink: int = 1, n_local: int = 1, k_min: int = 0, workspace=None, stream=None):
    """One decode step: (stats, if not given) -> selection -> sparse decode attention."""
    T = kc.shape[2]
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    if mean is None or var is None:
        mean, var = spa_block_stats(kc, block, stream=stream)
    idx, count = spa_select(q, mean, var, T, block, scale, top_p, n_sink, n_local, k_min,
                            stream=stream)
    out = spa_sparse_attn_decode(q, kc, vc, block, idx, count, scale, workspace=workspace,
                                 stream=stream)
    return {"out": out, "idx": idx, "count": count, "mean": mean, "var": var}


def decode_tree(q, kc, vc, parents, block: int, top_p: float, mean=None, var=None,
                scale: float | None = None, n_sink: int = 1, n_local: int = 1, k_min: int = 0,
                workspace=None, want_lse: bool = False, stream=None):
    """One step over a tree of n drafted tokens, in the last n rows of the caches: (stats, if
    not given) -> selection by node 0's query -> tree attention over the kept blocks.

    The T - n rows before the tree are the committed text, and the selection is of their
    blocks alone: the last n_local of them are kept, and the drafted rows, which the tree
    attends to anyway, take no part. mean and var are the statistics of those rows' blocks
    (more blocks may follow: they are not read). The tree of one node is a decode step:
    selected as by decode(), over all T rows.
    Returns dict(out, lse, idx, count, mean, var), mean and var those of the selection.
    """
    B, Hq, n, d = q.shape
    Hkv, T = kc.shape[1], kc.shape[2]
    text = T if n == 1 else max(T - n, 0)
    nb, cap = -(-text // block), -(-T // block)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    with _On(q, stream):
        if mean is None or var is None:
            whole = text // block if text < T else cap           # blocks without a drafted row
            mean, var = spa_block_stats(kc, block, 0, whole)
            if whole < nb:                                       # the text's last block, cut at its end
                tail = spa_block_stats(kc[:, :, whole * block:text].contiguous(), block)
                mean[:, :, whole:nb], var[:, :, whole:nb] = tail
        elif mean.shape[2] < nb or var.shape[2] < nb:
            raise ValueError(f"mean and var must hold the {nb} blocks of the {text} rows before the tree")
        mean, var = mean[:, :, :nb].contiguous(), var[:, :, :nb].contiguous()
        if text > 0:
            idx, count = spa_select(q[:, :, :1].contiguous(), mean, var, text, block, scale, top_p, n_sink,
                                    n_local, k_min, cap=cap)
        else:
            idx = torch.zeros((B, Hq, 1, cap), device=q.device, dtype=torch.int32)
            count = torch.zeros((B, Hq, 1), device=q.device, dtype=torch.int32)
        out, lse = spa_sparse_attn_tree(q, kc, vc, parents, block, idx, count, scale,
                                        workspace=workspace, want_lse=want_lse)
    return {"out": out, "lse": lse, "idx": idx, "count": count, "mean": mean, "var": var}


def evict(kc, vc, score, n_keep: int, n_sink: int = 4, n_recent: int = 0, lens=None, stream=None):
    """A smaller cache of the n_keep keys per kv-head with the most accumulated attention
    weight: choice -> move.

    Returns dict(k, v, score, keep, count).
    """
    keep, count = spa_evict_select(score, n_keep, n_sink, n_recent, lens=lens, stream=stream)
    k, v, score = spa_cache_gather(kc, vc, keep, count, score=score, stream=stream)
    return {"k": k, "v": v, "score": score, "keep": keep, "count": count}

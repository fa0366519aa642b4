"""The paged cache of 4-bit values: appending to it, attention over it, and what it
holds as numbers.

The cache is two uint8 tensors [num_pages, Hkv, page_size * (D / 2 + D / 32)] (see
fp4_cache; the layout of a page is described in include/dflash2.h); tables, lengths
and token rows are those of `target`, and so are the prepared calls.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import PagedKv, _dev, _dtype_code, load
from .target import _int32, _ints, _Prepared, _rows


def fp4_page_bytes(page_size: int, D: int) -> int:
    """Bytes of one head of a page: codes, then scales."""
    return page_size * (D // 2 + D // 32)


def fp4_cache(num_pages: int, Hkv: int, page_size: int, D: int, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """An empty cache (keys, values), all of it zeros."""
    shape = (num_pages, Hkv, fp4_page_bytes(page_size, D))
    return tuple(torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))


def _fp4_pages(k_cache: torch.Tensor, v_cache: torch.Tensor, D: int) -> Tuple[int, int, int, int]:
    """(pages, Hkv, page_size, page stride in bytes) of a 4-bit cache."""
    if k_cache.dim() != 3 or k_cache.shape != v_cache.shape or k_cache.dtype != torch.uint8 or v_cache.dtype != torch.uint8:
        raise ValueError("k_cache and v_cache must be uint8 [num_pages, Hkv, page_size * (D / 2 + D / 32)]")
    pages, Hkv, size = k_cache.shape
    row = D // 2 + D // 32
    if D % 32 or D < 32 or size % row:
        raise ValueError("%d bytes of a head of a page are no rows of head size %d" % (size, D))
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_cuda:
            raise ValueError("%s must be a GPU tensor" % name)
        if t.numel() and ((Hkv > 1 and t.stride(1) != size) or (size > 1 and t.stride(2) != 1)):
            raise ValueError("%s: a page must be contiguous" % name)
    if pages > 1 and k_cache.stride(0) != v_cache.stride(0):
        raise ValueError("k_cache and v_cache must have one page stride")
    _int32(num_pages=pages, Hkv=Hkv, page_size=size // row)
    return pages, Hkv, size // row, k_cache.stride(0) if pages > 1 else Hkv * size


def _fp4_descriptor(k_cache, v_cache, block_table, ctx_len, tok_start, N: int, Hq: int, D: int, rows: torch.Tensor) -> PagedKv:
    pages, Hkv, page, stride = _fp4_pages(k_cache, v_cache, D)
    B = ctx_len.shape[0] if ctx_len.dim() == 1 else -1
    _ints(ctx_len, "ctx_len", (B,))
    _ints(tok_start, "tok_start", (B + 1,))
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != B:
        raise ValueError("block_table must be int32 [B, pages of a sequence]")
    width = block_table.shape[1]
    if not block_table.is_cuda:
        raise ValueError("block_table must be a GPU tensor")
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: a sequence's row must be contiguous")
    _int32(N=N, table_width=width)
    return PagedKv(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), _dev(ctx_len, "ctx_len"),
                   _dev(tok_start, "tok_start"), stride, block_table.stride(0) if B > 1 else width, B, N, Hq, Hkv, D, page,
                   pages, width, _dtype_code(rows))


class PreparedAppendFp4(_Prepared):
    """dflash2_kv_append_fp4: as PreparedAppend, into a 4-bit cache (k_cache, v_cache
    uint8 [num_pages, Hkv, page_size * (D / 2 + D / 32)])."""

    def __init__(self, k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q: Optional[torch.Tensor] = None,
                 q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 rope_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                 out_q: Optional[torch.Tensor] = None):
        lib = load()
        if k.dim() != 3:
            raise ValueError("k must be [N, Hkv, D]")
        N, D, dt = k.shape[0], k.shape[2], k.dtype
        Hq = q.shape[1] if q is not None else k.shape[1]
        self.kv = kv = _fp4_descriptor(k_cache, v_cache, block_table, ctx_len, tok_start, N, Hq, D, k)
        strides = [0, _rows(k, "k", N, kv.Hkv, D, dt), _rows(v, "v", N, kv.Hkv, D, dt), 0]
        if q is not None:
            strides[0] = _rows(q, "q", N, Hq, D, dt)
            if out_q is None:
                out_q = torch.empty((N, Hq, D), dtype=dt, device=q.device)
            strides[3] = _rows(out_q, "out_q", N, Hq, D, dt)
        elif out_q is not None:
            raise ValueError("out_q without q")
        for name, t in (("q_norm", q_norm), ("k_norm", k_norm)):
            if t is not None and (t.dtype != dt or tuple(t.shape) != (D,)):
                raise ValueError("%s must be [%d] in the dtype of k" % (name, D))
        if rope_freq is not None and (rope_freq.dtype != torch.float64 or rope_freq.dim() != 1):
            raise ValueError("rope_freq must be float64 [rot / 2]")
        rot = 0 if rope_freq is None else 2 * rope_freq.shape[0]

        def at(t):
            return t.data_ptr() if t is not None else None

        args = (ctypes.byref(kv), at(q), strides[0], at(k), strides[1], at(v), strides[2],
                _dev(q_norm, "q_norm") if q_norm is not None else None,
                _dev(k_norm, "k_norm") if k_norm is not None else None, float(eps),
                _dev(rope_freq, "rope_freq") if rope_freq is not None else None, rot, int(interleaved),
                at(out_q), strides[3])
        self._ready(lib.dflash2_kv_append_fp4, args, k_cache.device,
                    (k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q, q_norm, k_norm, rope_freq, out_q),
                    out_q)


class PreparedAttentionFp4(_Prepared):
    """dflash2_paged_attention_fp4: as PreparedAttention, over a 4-bit cache (k_cache,
    v_cache uint8 [num_pages, Hkv, page_size * (D / 2 + D / 32)])."""

    def __init__(self, q, k_cache, v_cache, block_table, ctx_len, tok_start, scale: Optional[float] = None,
                 causal: bool = True, window: int = 0, max_len: Optional[int] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        lib = load()
        length = min(int(max_len), 2**31 - 1) if max_len is not None else 0
        _int32(window=int(window), max_len=length)
        if q.dim() != 3:
            raise ValueError("q must be [N, Hq, D]")
        N, Hq, D = q.shape
        self.kv = kv = _fp4_descriptor(k_cache, v_cache, block_table, ctx_len, tok_start, N, Hq, D, q)
        q_stride = _rows(q, "q", N, Hq, D, q.dtype)
        if out is None:
            out = torch.empty((N, Hq, D), dtype=q.dtype, device=q.device)
        out_stride = _rows(out, "out", N, Hq, D, q.dtype)
        need = lib.dflash2_paged_attention_fp4_workspace(ctypes.byref(kv), length)
        if workspace is None:
            workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
        elif workspace.dtype != torch.uint8:
            raise ValueError("workspace must be uint8")
        args = (ctypes.byref(kv), q.data_ptr(), q_stride, float(D ** -0.5 if scale is None else scale),
                int(causal), int(window), length, out.data_ptr(), out_stride,
                _dev(workspace, "workspace") if workspace.numel() else None, workspace.numel())
        self._ready(lib.dflash2_paged_attention_fp4, args, k_cache.device,
                    (q, k_cache, v_cache, block_table, ctx_len, tok_start, out, workspace), out)


class PreparedUnpackFp4(_Prepared):
    """dflash2_kv_unpack_fp4: what all pages of a 4-bit cache of head size D hold.
    Calling it returns (keys, values) [num_pages, Hkv, page_size, D] in `dtype`, a cache
    as paged_attention takes it."""

    def __init__(self, k_cache, v_cache, D: int, dtype: torch.dtype = torch.bfloat16,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
        lib = load()
        pages, Hkv, page, stride = _fp4_pages(k_cache, v_cache, D)
        shape = (pages, Hkv, page, D)
        if out is None:
            out = tuple(torch.empty(shape, dtype=dtype, device=k_cache.device) for _ in range(2))
        for t in out:
            if tuple(t.shape) != shape or t.dtype != dtype:
                raise ValueError("out must be two tensors %s of %s" % (list(shape), dtype))
        self.kv = kv = PagedKv(k_cache.data_ptr(), v_cache.data_ptr(), None, None, None, stride, 1, 0, 0, Hkv, Hkv, D, page,
                               pages, 1, _dtype_code(out[0]))
        args = (ctypes.byref(kv), _dev(out[0], "out"), _dev(out[1], "out"))
        self._ready(lib.dflash2_kv_unpack_fp4, args, k_cache.device, (k_cache, v_cache) + tuple(out), tuple(out))


def kv_append_fp4(k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q=None, q_norm=None, k_norm=None,
                  eps: float = 1e-6, rope_freq=None, interleaved: bool = False, out_q=None) -> Optional[torch.Tensor]:
    """New keys and values into the 4-bit cache, queries and keys normed and rotated on
    the way (see PreparedAppendFp4): the queries, or None without q."""
    return PreparedAppendFp4(k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q, q_norm, k_norm, eps, rope_freq,
                             interleaved, out_q)()


def paged_attention_fp4(q, k_cache, v_cache, block_table, ctx_len, tok_start, scale: Optional[float] = None,
                        causal: bool = True, window: int = 0, max_len: Optional[int] = None,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the new tokens over their sequences' positions in a 4-bit cache (see
    PreparedAttentionFp4): [N, Hq, D]."""
    return PreparedAttentionFp4(q, k_cache, v_cache, block_table, ctx_len, tok_start, scale, causal, window, max_len,
                                out)()


def kv_unpack_fp4(k_cache, v_cache, D: int, dtype: torch.dtype = torch.bfloat16) -> Tuple[torch.Tensor, torch.Tensor]:
    """What a 4-bit cache holds (see PreparedUnpackFp4): (keys, values)."""
    return PreparedUnpackFp4(k_cache, v_cache, D, dtype)()

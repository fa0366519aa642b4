"""Between the steps of a serving loop: the pages, token starts and slots of the
next step from the lengths of the requests, and the penalties, biases and masks on
the target's rows before they are verified.

Prepared calls and functions as in `target`; the arithmetic is in the HIP kernels
(include/dflash2.h).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import Adjust, PagePool, _dev, _dtype_code, load
from .target import _int32, _ints, _Prepared


def _pointer(t: Optional[torch.Tensor], name: str):
    return _dev(t, name) if t is not None else None


class PreparedPages(_Prepared):
    """dflash2_plan_pages: block_table [B, width], held [B], free_list [num_pages] and
    free_count [1] (int32, updated in place) brought to what B requests of ctx_len [B]
    tokens want that were joined by advance [B] and bring n_new [B] (negative: ended);
    rows: token rows of the step.  Calling it returns (tok_start [B + 1], ctx_out [B],
    slots [rows] int64, positions [rows] int32); ctx_out may be ctx_len itself."""

    def __init__(self, block_table, held, free_list, free_count, ctx_len, n_new, page_size: int, rows: int,
                 advance: Optional[torch.Tensor] = None, ctx_out: Optional[torch.Tensor] = None):
        lib = load()
        if block_table.dim() != 2 or block_table.dtype != torch.int32:
            raise ValueError("block_table must be int32 [B, pages of a request]")
        B, width = block_table.shape
        if not block_table.is_cuda:
            raise ValueError("block_table must be a GPU tensor")
        if width > 1 and block_table.stride(1) != 1:
            raise ValueError("block_table: a request's row must be contiguous")
        if rows < 0:
            raise ValueError("rows must be >= 0")
        _int32(rows=int(rows), page_size=int(page_size))
        if free_list.dim() != 1:
            raise ValueError("free_list must be int32 [pages of the cache]")
        pages = free_list.shape[0]
        _int32(num_pages=pages, table_width=width, B=B)
        for t, name, shape in ((held, "held", (B,)), (free_list, "free_list", (pages,)), (free_count, "free_count", (1,)),
                               (ctx_len, "ctx_len", (B,)), (n_new, "n_new", (B,)), (advance, "advance", (B,)),
                               (ctx_out, "ctx_out", (B,))):
            if t is not None:
                _ints(t, name, shape)
        dev = block_table.device
        if ctx_out is None:
            ctx_out = torch.empty((B,), dtype=torch.int32, device=dev)
        start = torch.empty((B + 1,), dtype=torch.int32, device=dev)
        slots = torch.empty((rows,), dtype=torch.int64, device=dev)
        positions = torch.empty((rows,), dtype=torch.int32, device=dev)
        self._pool = pool = PagePool(block_table.data_ptr(), _dev(held, "held"), _dev(free_list, "free_list"),
                                     _dev(free_count, "free_count"), block_table.stride(0) if B > 1 else width, B,
                                     int(rows), int(page_size), pages, width)
        args = (ctypes.byref(pool), _dev(ctx_len, "ctx_len"), _pointer(advance, "advance"), _dev(n_new, "n_new"),
                _dev(ctx_out, "ctx_out"), start.data_ptr(), slots.data_ptr() if rows else None,
                positions.data_ptr() if rows else None)
        self._ready(lib.dflash2_plan_pages, args, dev,
                    (block_table, held, free_list, free_count, ctx_len, n_new, advance, ctx_out, start, slots, positions),
                    (start, ctx_out, slots, positions))


class PreparedAdjust(_Prepared):
    """dflash2_adjust_logits: rows logits [B, R, V] with penalties for the tokens of
    history [B, L] (its first history_len [B], of which prompt_len [B] are the prompt)
    and of the drafts path [B, R - 1] before a row (repetition, frequency, presence
    [B] float32), biases bias [B, M] float32 on bias_token [B, M] (a token given twice:
    the last), and -inf where mask [B, R, ceil(V / 32)] (int32 words, bit v % 32 of word
    v / 32; B and R may be broadcast) has no bit.  out: where they go, logits itself for
    in place (default: a new tensor).  Calling it returns out."""

    def __init__(self, logits, history: Optional[torch.Tensor] = None, history_len: Optional[torch.Tensor] = None,
                 prompt_len: Optional[torch.Tensor] = None, path: Optional[torch.Tensor] = None,
                 repetition: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                 presence: Optional[torch.Tensor] = None, bias_token: Optional[torch.Tensor] = None,
                 bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None):
        lib = load()
        if logits.dim() != 3:
            raise ValueError("logits must be [B, R, V]")
        B, R, V = logits.shape
        _int32(B=B, R=R, V=V)
        dt = _dtype_code(logits)
        if out is None:
            out = torch.empty((B, R, V), dtype=logits.dtype, device=logits.device)
        elif out.dtype != logits.dtype or out.shape != logits.shape:
            raise ValueError("out must have the shape and dtype of logits")
        for name, t in (("logits", logits), ("out", out)):
            if not t.is_cuda:
                raise ValueError("%s must be a GPU tensor" % name)
            if V > 1 and t.stride(2) != 1:
                raise ValueError("%s: a row must be contiguous" % name)
        L = M = words = 0
        if (history is None) != (history_len is None):
            raise ValueError("history and history_len come together")
        if history is not None:
            if history.dim() != 2 or history.dtype != torch.int32 or history.shape[0] != B:
                raise ValueError("history must be int32 [B, tokens]")
            if not history.is_cuda:
                raise ValueError("history must be a GPU tensor")
            L = history.shape[1]
            if L > 1 and history.stride(1) != 1:
                raise ValueError("history: a sequence's row must be contiguous")
            _ints(history_len, "history_len", (B,))
        elif prompt_len is not None:
            raise ValueError("prompt_len without history")
        if prompt_len is not None:
            _ints(prompt_len, "prompt_len", (B,))
        if path is not None:
            _ints(path, "path", (B, max(R - 1, 0)))
        for name, t in (("repetition", repetition), ("frequency", frequency), ("presence", presence)):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (B,)):
                raise ValueError("%s must be float32 [%d]" % (name, B))
        if (bias_token is None) != (bias is None):
            raise ValueError("bias_token and bias come together")
        if bias is not None:
            if bias.dim() != 2:
                raise ValueError("bias must be float32 [B, biases]")
            M = bias.shape[1]
            if bias.dtype != torch.float32 or tuple(bias.shape) != (B, M):
                raise ValueError("bias must be float32 [%d, %d]" % (B, M))
            _ints(bias_token, "bias_token", (B, M))
        if mask is not None:
            words = (V + 31) // 32
            _ints(mask, "mask", (B, R, words))
            if not mask.is_cuda:
                raise ValueError("mask must be a GPU tensor")
            if words > 1 and mask.stride(2) != 1:
                raise ValueError("mask: a row must be contiguous")
        _int32(L=L, M=M)

        def at(t, name):
            return _pointer(t, name) if t is not None and t.numel() else None

        def strides(t):
            # of sequences and rows; one that is never stepped by may be anything
            row = t.stride(1) if R > 1 else V
            return (t.stride(0) if B > 1 else max(R - 1, 0) * row + V), row

        self._adjust = a = Adjust(B, R, V, L, M, dt, *strides(logits), *strides(out),
                                  history.data_ptr() if L and B else None,
                                  (history.stride(0) if B > 1 else L) if L else 0,
                                  *(at(t, n) for t, n in ((history_len, "history_len"), (prompt_len, "prompt_len"),
                                                          (path, "path"), (repetition, "repetition"),
                                                          (frequency, "frequency"), (presence, "presence"),
                                                          (bias_token, "bias_token"), (bias, "bias"))),
                                  mask.data_ptr() if words else None, mask.stride(0) if words and B > 1 else 0,
                                  mask.stride(1) if words and R > 1 else 0)
        self._ready(lib.dflash2_adjust_logits, (ctypes.byref(a), logits.data_ptr(), out.data_ptr()), logits.device,
                    (logits, history, history_len, prompt_len, path, repetition, frequency, presence, bias_token, bias,
                     mask, out), out)


def plan_pages(block_table, held, free_list, free_count, ctx_len, n_new, page_size: int, rows: int,
               advance=None, ctx_out=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """The pages of the next step (see PreparedPages): (tok_start, ctx_out, slots,
    positions); block_table, held, free_list and free_count are updated."""
    return PreparedPages(block_table, held, free_list, free_count, ctx_len, n_new, page_size, rows, advance, ctx_out)()


def adjust_logits(logits, history=None, history_len=None, prompt_len=None, path=None, repetition=None, frequency=None,
                  presence=None, bias_token=None, bias=None, mask=None, out=None) -> torch.Tensor:
    """Rows of logits with penalties, biases and masks (see PreparedAdjust)."""
    return PreparedAdjust(logits, history, history_len, prompt_len, path, repetition, frequency, presence, bias_token,
                          bias, mask, out)()

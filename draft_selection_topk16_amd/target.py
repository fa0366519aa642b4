"""The target's side of a draft-verify cycle: new tokens into a paged key/value
cache, their attention over it, and the verification of drafted tokens.

Each operator has a prepared call, whose arguments are checked once and which
then enqueues with little host work on the stream that is current when it is
called, and a function that prepares and calls.  Refill the tensors of a
prepared call in place between calls; calls of one prepared call (and replays
of graphs that captured it) share its outputs and workspace and must be
ordered.  It may be dropped while it still runs on any stream that it was called
on, but must be kept as long as a graph that captured it is replayed.  The
arithmetic is in the HIP kernels (include/dflash2.h).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import PagedKv, VerifyDims, _check, _dev, _dtype_code, load

TARGET_KINDS = {"logits": 0, "probs": 1}


# The current device and stream as numbers: the objects torch makes of a stream
# take longer (2.6 us) than a launch.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _Prepared:
    """A checked call: its arguments but the stream, and what it keeps alive."""

    def _ready(self, fn, args, device: torch.device, keep, out) -> None:
        for t in keep:
            if t is not None and t.device != device:
                raise ValueError("every tensor must be on %s" % device)
        # converted once: ctypes then passes them as they are
        self._args = tuple(a if isinstance(a, ctypes._SimpleCData) or hasattr(a, "_obj") else kind(a)
                           for a, kind in zip(args, fn.argtypes))
        self._fn, self._keep, self._out = fn, keep, out
        self._index = device.index if device.index is not None else torch.cuda.current_device()
        self._streams = {_raw_stream(self._index)}      # that the allocator knows to use the tensors

    def _use_on(self, index: int, stream: int) -> None:
        """Tells the allocator of another stream than the one that the tensors were made
        on: their memory is not given away while a call runs there."""
        current = torch.cuda.current_stream(index)
        for t in self._keep:
            if t is not None:
                t.record_stream(current)
        self._streams.add(stream)

    def __call__(self):
        index = self._index
        stream = _raw_stream(index)
        if stream not in self._streams:
            self._use_on(index, stream)
        if _current_device() == index:
            status = self._fn(*self._args, stream)
        else:
            with torch.cuda.device(index):
                status = self._fn(*self._args, stream)
        if status:
            _check(status)
        return self._out


def _int32(**sizes: int) -> None:
    """ctypes would cut a larger number down to 32 bits."""
    for name, x in sizes.items():
        if not -2**31 <= x < 2**31:
            raise ValueError("%s = %d does not fit 32 bits" % (name, x))


def _ints(t: torch.Tensor, name: str, shape) -> torch.Tensor:
    if t.dtype != torch.int32 or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be int32 %s" % (name, list(shape)))
    return t


def _rows(t: torch.Tensor, name: str, N: int, H: int, D: int, dtype: torch.dtype) -> int:
    """The token stride of [N, H, D] rows whose heads follow one another."""
    if t.dtype != dtype:
        raise TypeError("%s must have the cache's dtype" % name)
    if tuple(t.shape) != (N, H, D):
        raise ValueError("%s must be [%d, %d, %d]" % (name, N, H, D))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.numel() and ((D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D)):
        raise ValueError("%s: a token's heads must be contiguous" % name)
    return t.stride(0) if N > 1 else H * D


def _descriptor(k_cache, v_cache, block_table, ctx_len, tok_start, N: int, Hq: int) -> PagedKv:
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.dtype != v_cache.dtype:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, D] of one dtype")
    pages, Hkv, page, D = k_cache.shape
    dense = (Hkv * page * D, page * D, D, 1)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not t.is_cuda:
            raise ValueError("%s must be a GPU tensor" % name)
        if t.numel() and any(n > 1 and s != d for n, s, d in zip(t.shape[1:], t.stride()[1:], dense[1:])):
            raise ValueError("%s: a page must be contiguous" % name)
    if pages > 1 and k_cache.stride(0) != v_cache.stride(0):
        raise ValueError("k_cache and v_cache must have one page stride")
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
    _int32(N=N, num_pages=pages, table_width=width)
    return PagedKv(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), _dev(ctx_len, "ctx_len"),
                   _dev(tok_start, "tok_start"), k_cache.stride(0) if pages > 1 else dense[0],
                   block_table.stride(0) if B > 1 else width, B, N, Hq, Hkv, D, page, pages, width,
                   _dtype_code(k_cache))


def rope_freqs(rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """base^(-2i / rot), i = 0 .. rot / 2 - 1, float64: radians a position of each pair."""
    return float(base) ** (-torch.arange(rot // 2, dtype=torch.float64, device=device) * 2.0 / rot)


class PreparedAppend(_Prepared):
    """dflash2_kv_append: k, v [N, Hkv, D] of the new tokens into the paged cache
    (k_cache, v_cache [num_pages, Hkv, page_size, D], block_table [B, width],
    ctx_len [B] tokens before, tok_start [B + 1]); queries and keys normed per
    head (q_norm, k_norm [D]) and rotated (rope_freq [rot / 2] float64).
    Calling it returns out_q [N, Hq, D], or None without q; out_q may be q."""

    def __init__(self, k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q: Optional[torch.Tensor] = None,
                 q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 rope_freq: Optional[torch.Tensor] = None, interleaved: bool = False,
                 out_q: Optional[torch.Tensor] = None):
        lib = load()
        N, Hq = k.shape[0], (q.shape[1] if q is not None else k.shape[1])
        self.kv = kv = _descriptor(k_cache, v_cache, block_table, ctx_len, tok_start, N, Hq)
        dt, D = k_cache.dtype, kv.D
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
                raise ValueError("%s must be [%d] in the cache's dtype" % (name, D))
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
        self._ready(lib.dflash2_kv_append, args, k_cache.device,
                    (k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q, q_norm, k_norm, rope_freq, out_q),
                    out_q)


class PreparedAttention(_Prepared):
    """dflash2_paged_attention: q [N, Hq, D] of the new tokens over the paged cache
    (arguments as for PreparedAppend); scale defaults to D^-1/2.  max_len: an
    upper estimate of ctx_len + new tokens for the launch plan (default: what
    block_table can hold).  Calling it returns out [N, Hq, D]."""

    def __init__(self, q, k_cache, v_cache, block_table, ctx_len, tok_start, scale: Optional[float] = None,
                 causal: bool = True, window: int = 0, max_len: Optional[int] = None,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        lib = load()
        length = min(int(max_len), 2**31 - 1) if max_len is not None else 0
        _int32(window=int(window), max_len=length)
        N, Hq, D = q.shape
        self.kv = kv = _descriptor(k_cache, v_cache, block_table, ctx_len, tok_start, N, Hq)
        dt = k_cache.dtype
        if D != kv.D:
            raise ValueError("q and the cache disagree on D")
        q_stride = _rows(q, "q", N, Hq, D, dt)
        if out is None:
            out = torch.empty((N, Hq, D), dtype=dt, device=q.device)
        out_stride = _rows(out, "out", N, Hq, D, dt)
        need = lib.dflash2_paged_attention_workspace(ctypes.byref(kv), length)
        if workspace is None:
            workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
        elif workspace.dtype != torch.uint8:
            raise ValueError("workspace must be uint8")
        args = (ctypes.byref(kv), q.data_ptr(), q_stride, float(D ** -0.5 if scale is None else scale),
                int(causal), int(window), length, out.data_ptr(), out_stride,
                _dev(workspace, "workspace") if workspace.numel() else None, workspace.numel())
        self._ready(lib.dflash2_paged_attention, args, k_cache.device,
                    (q, k_cache, v_cache, block_table, ctx_len, tok_start, out, workspace), out)


class PreparedVerify(_Prepared):
    """dflash2_verify: the drafted path [B, P] against target rows [B, P + 1, V]
    (kind "logits", at a temperature, or "probs"), the draft's distributions
    prob [B, P, K] over cand [B, P, K], uniforms u [B, P + 1]; n_draft [B] int32
    drafts in use.  At temperature 0 cand, prob and u may be None.  Calling it
    returns (tokens [B, P + 1] int32, count [B] int32, p [B, P + 1] float32)."""

    def __init__(self, target, path, cand: Optional[torch.Tensor], prob: Optional[torch.Tensor],
                 u: Optional[torch.Tensor], temperature: float = 1.0, n_draft: Optional[torch.Tensor] = None,
                 kind: str = "logits", workspace: Optional[torch.Tensor] = None):
        lib = load()
        if kind not in TARGET_KINDS:
            raise ValueError("kind must be one of %s" % sorted(TARGET_KINDS))
        if target.dim() != 3 or target.shape[1] < 2:
            raise ValueError("target must be [B, P + 1, V]")
        B, P, V = target.shape[0], target.shape[1] - 1, target.shape[2]
        _int32(B=B, V=V)
        _ints(path, "path", (B, P))
        K = 1
        if cand is not None:
            if cand.dim() != 3:
                raise ValueError("cand must be int32 [B, P, K]")
            K = cand.shape[2]
            _ints(cand, "cand", (B, P, K))
        for name, t, shape in (("prob", prob, (B, P, K)), ("u", u, (B, P + 1))):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape):
                raise ValueError("%s must be float32 %s" % (name, list(shape)))
        if n_draft is not None:
            _ints(n_draft, "n_draft", (B,))
        self._dims = dims = VerifyDims(B, P, V, K, _dtype_code(target), TARGET_KINDS[kind])
        at = {n: _dev(t, n) if t is not None else None
              for n, t in (("target", target), ("path", path), ("cand", cand), ("prob", prob), ("n_draft", n_draft),
                           ("u", u))}
        need = lib.dflash2_verify_workspace(ctypes.byref(dims))
        if workspace is None:
            workspace = torch.empty((need,), dtype=torch.uint8, device=target.device)
        elif workspace.dtype != torch.uint8:
            raise ValueError("workspace must be uint8")
        tok = torch.empty((B, P + 1), dtype=torch.int32, device=target.device)
        count = torch.empty((B,), dtype=torch.int32, device=target.device)
        p = torch.empty((B, P + 1), dtype=torch.float32, device=target.device)
        args = (ctypes.byref(dims), at["target"], at["path"], at["cand"], at["prob"], at["n_draft"],
                float(temperature), at["u"], tok.data_ptr(), count.data_ptr(), p.data_ptr(),
                _dev(workspace, "workspace") if workspace.numel() else None, workspace.numel())
        self._ready(lib.dflash2_verify, args, target.device,
                    (target, path, cand, prob, u, n_draft, workspace, tok, count, p), (tok, count, p))


def kv_append(k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q=None, q_norm=None, k_norm=None,
              eps: float = 1e-6, rope_freq=None, interleaved: bool = False, out_q=None) -> Optional[torch.Tensor]:
    """New keys and values into the paged cache, queries and keys normed and
    rotated on the way (see PreparedAppend): the queries, or None without q."""
    return PreparedAppend(k, v, k_cache, v_cache, block_table, ctx_len, tok_start, q, q_norm, k_norm, eps, rope_freq,
                          interleaved, out_q)()


def paged_attention(q, k_cache, v_cache, block_table, ctx_len, tok_start, scale: Optional[float] = None,
                    causal: bool = True, window: int = 0, max_len: Optional[int] = None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the new tokens over their sequences' cached positions (see
    PreparedAttention): [N, Hq, D]."""
    return PreparedAttention(q, k_cache, v_cache, block_table, ctx_len, tok_start, scale, causal, window, max_len,
                             out)()


def verify(target, path, cand=None, prob=None, u=None, temperature: float = 1.0, n_draft=None,
           kind: str = "logits") -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Which drafted tokens stand, and the next token (see PreparedVerify):
    (tokens [B, P + 1] int32 with -1 behind the last, count [B] int32, p)."""
    return PreparedVerify(target, path, cand, prob, u, temperature, n_draft, kind)()

"""Both ends of a language model: embedding lookup and its gradient, dropout,
and softmax cross entropy against the vocabulary table. Gradients of tables go
straight into the tensor's place in a flat gradient vector.

As in the rest of the binding: checks and marshalling, the work runs in the
library's kernels on the current stream of the tensors' device (or `stream`).
Results and workspaces come from torch's allocator on that stream, so a call
can be captured in a graph.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _check, _dtype_code, _stream_handle, _torch_stream, lib


class _Drop(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("counter", ctypes.c_void_p)]


_declared = None


def _lib():
    global _declared
    L = lib()
    if _declared is not L:
        i64, i32, vp, dbl, dt = (ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_double,
                                 ctypes.c_int)
        p64, pdrop = ctypes.POINTER(i64), ctypes.POINTER(_Drop)
        L.zero_embed.argtypes = [vp, i32, i64, vp, i64, i64, dt, dbl, vp, vp, i64, pdrop, vp, dt, vp]
        L.zero_embed_grad_workspace.argtypes = [i64, i64, i64, p64]
        L.zero_embed_grad.argtypes = [vp, dt, vp, i32, i64, i64, i64, dbl, pdrop, vp, dt, i32, vp,
                                      i64, vp]
        L.zero_dropout.argtypes = [vp, vp, vp, i64, dt, pdrop, vp]
        L.zero_head_loss_workspace.argtypes = [i64, i64, i64, dt, i32, i32, dt, i64, p64]
        L.zero_head_loss.argtypes = [vp, vp, dt, vp, i32, i64, i64, i64, vp, i32, dbl, vp, vp, vp,
                                     vp, dt, i32, i64, vp, i64, vp]
        _declared = L
    return L


@dataclass(frozen=True)
class Dropout:
    """Which elements dropout drops: probability p (taken to a multiple of
    2^-16), and the counter-based generator's seed and offset, 64 bits each.
    The forward and the backward call of one place take the same; other steps
    and layers other offsets. counter: one int64 on the device, added to offset
    when the kernel runs, for steps replayed from a graph."""
    p: float
    seed: int
    offset: int = 0
    counter: Optional[torch.Tensor] = None

    def _struct(self, device: torch.device) -> _Drop:
        if not 0 <= self.seed < 1 << 64 or not 0 <= self.offset < 1 << 64:
            raise ValueError("seed and offset must be in [0, 2^64)")
        c = self.counter
        if c is not None and (c.device != device or c.dtype != torch.int64 or c.numel() != 1):
            raise ValueError(f"counter must be one int64 on {device}")
        return _Drop(float(self.p), self.seed, self.offset, None if c is None else c.data_ptr())


class _Call:
    """The device and stream of one call, and checks of its tensors."""

    def __init__(self, first: torch.Tensor, what: str, stream):
        if first.device.type != "cuda":
            raise ValueError(f"{what} must be on a cuda device, got {first.device}")
        self.device, self.stream = first.device, stream
        self.handle = _stream_handle(stream, self.device)
        self._scopes = None

    def __enter__(self):
        if self.stream is not None or torch.cuda.current_device() != self.device.index:
            self._scopes = contextlib.ExitStack()
            self._scopes.enter_context(torch.cuda.device(self.device))
            if self.stream is not None:
                self._scopes.enter_context(
                    torch.cuda.stream(_torch_stream(self.stream, self.device)))
        return self

    def __exit__(self, *exc):
        if self._scopes is not None:
            self._scopes.close()

    def ptr(self, x: Optional[torch.Tensor], what: str, dtype=None, shape=None, numel=None):
        """Address of a contiguous tensor on the call's device; None for None."""
        if x is None:
            return None
        if x.device != self.device:
            raise ValueError(f"{what} is on {x.device}, the call is on {self.device}")
        if not x.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        if dtype is not None and x.dtype != dtype:
            raise TypeError(f"{what} is {x.dtype}, need {dtype}")
        if shape is not None and x.shape != shape:
            raise ValueError(f"{what} has shape {tuple(x.shape)}, need {tuple(shape)}")
        if numel is not None and x.numel() != numel:
            raise ValueError(f"{what} has {x.numel()} elements, need {numel}")
        if self.stream is not None:
            x.record_stream(_torch_stream(self.stream, self.device))
        return x.data_ptr()

    def ids(self, x: torch.Tensor, what: str):
        """(address, bytes of an id)"""
        if x.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"{what} must be int32 or int64, got {x.dtype}")
        return self.ptr(x, what), x.element_size()

    def drop(self, d: Optional[Dropout]):
        if d is None:
            return None
        if d.counter is not None and self.stream is not None:
            d.counter.record_stream(_torch_stream(self.stream, self.device))
        return ctypes.byref(d._struct(self.device))

    def workspace(self, size, *args) -> torch.Tensor:
        n = ctypes.c_int64()
        _check(size(*args, ctypes.byref(n)))
        return torch.empty(n.value, dtype=torch.uint8, device=self.device)


def _table(x: torch.Tensor, what: str):
    if x.dim() != 2:
        raise ValueError(f"{what} must have two dimensions, got {tuple(x.shape)}")
    return x.shape


def embed(tokens: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0,
          positions: Optional[torch.Tensor] = None, position_table: Optional[torch.Tensor] = None,
          dropout: Optional[Dropout] = None, out: Optional[torch.Tensor] = None,
          dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """dropout(scale * table[tokens] + position_table[positions]), of shape
    tokens.shape + (width,). Ids outside a table give a row of zeros. The
    result is `out`, or a new tensor of `dtype` (the table's by default)."""
    rows, width = _table(table, "table")
    if (positions is None) != (position_table is None):
        raise ValueError("positions and position_table come together")
    with _Call(tokens, "tokens", stream) as c:
        shape = (*tokens.shape, width)
        if out is None:
            out = torch.empty(shape, dtype=dtype or table.dtype, device=c.device)
        elif dtype is not None and out.dtype != dtype:
            raise TypeError(f"out is {out.dtype}, dtype asks for {dtype}")
        ids, size = c.ids(tokens, "tokens")
        pos = ptable = None
        prows = 0
        if positions is not None:
            if _table(position_table, "position_table")[1] != width:
                raise ValueError("table and position_table differ in width")
            pos = c.ptr(positions, "positions", tokens.dtype, tokens.shape)
            ptable = c.ptr(position_table, "position_table", table.dtype)
            prows = position_table.shape[0]
        _check(_lib().zero_embed(ids, size, tokens.numel(), c.ptr(table, "table"), rows, width,
                                 _dtype_code(table.dtype), float(scale), pos, ptable, prows,
                                 c.drop(dropout), c.ptr(out, "out", shape=shape),
                                 _dtype_code(out.dtype), c.handle))
    return out


def embed_grad(grad_out: torch.Tensor, tokens: torch.Tensor, grad_table: torch.Tensor, *,
               scale: float = 1.0, dropout: Optional[Dropout] = None, accumulate: bool = False,
               stream=None) -> torch.Tensor:
    """The gradient of embed's table, written into grad_table (rows, width), a
    view of a flat gradient vector for instance, or added to the rows that
    tokens name. The gradient of its position table is embed_grad(grad_out,
    positions, grad_position_table, dropout=dropout)."""
    rows, width = _table(grad_table, "grad_table")
    with _Call(tokens, "tokens", stream) as c:
        n = tokens.numel()
        L = _lib()
        ids, size = c.ids(tokens, "tokens")
        g = c.ptr(grad_out, "grad_out", numel=n * width)
        t = c.ptr(grad_table, "grad_table")
        gdt, tdt = _dtype_code(grad_out.dtype), _dtype_code(grad_table.dtype)
        ws = c.workspace(L.zero_embed_grad_workspace, n, rows, width)
        _check(L.zero_embed_grad(g, gdt, ids, size, n, rows, width, float(scale), c.drop(dropout),
                                 t, tdt, int(bool(accumulate)), ws.data_ptr(), ws.numel(),
                                 c.handle))
    return grad_table


def dropout(x: torch.Tensor, drop: Dropout, *, add: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dropout(x), plus `add` if given; dropout(grad, drop) is its backward.
    out may be x or add."""
    with _Call(x, "x", stream) as c:
        if out is None:
            out = torch.empty_like(x, memory_format=torch.contiguous_format)
        _check(_lib().zero_dropout(c.ptr(x, "x"), c.ptr(add, "add", x.dtype, x.shape),
                                   c.ptr(out, "out", x.dtype, x.shape), x.numel(),
                                   _dtype_code(x.dtype), c.drop(drop), c.handle))
    return out


def head_loss(hidden: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, *,
              weights: Optional[torch.Tensor] = None, reduction: str = "mean",
              grad_scale: float = 1.0, losses: Optional[torch.Tensor] = None,
              grad_hidden: Optional[torch.Tensor] = None,
              grad_table: Optional[torch.Tensor] = None, accumulate: bool = False,
              piece_rows: int = 0, stream=None) -> torch.Tensor:
    """Softmax cross entropy of hidden (..., width) against table (vocab,
    width) at targets (...), as one float32 on the device: the sum over rows of
    weight times loss, divided by the sum of the weights with "mean". Rows
    whose target is outside the table, or whose weight is 0, take no part.

    Written where given: losses (each row's), grad_hidden, and grad_table
    (bf16 or fp32, a view of a flat gradient vector for instance; added to with
    `accumulate`), the gradients of grad_scale * loss. The logits are never
    kept; piece_rows bounds the rows worked on at once (0: by memory)."""
    if reduction not in ("mean", "sum"):
        raise ValueError(f"reduction must be 'mean' or 'sum', got {reduction!r}")
    vocab, width = _table(table, "table")
    with _Call(hidden, "hidden", stream) as c:
        L, n = _lib(), targets.numel()
        if hidden.shape != (*targets.shape, width):
            raise ValueError(f"hidden has shape {tuple(hidden.shape)}, need "
                             f"{(*targets.shape, width)}")
        ids, size = c.ids(targets, "targets")
        h, t = c.ptr(hidden, "hidden"), c.ptr(table, "table", hidden.dtype)
        w = c.ptr(weights, "weights", torch.float32, targets.shape)
        ls = c.ptr(losses, "losses", torch.float32, targets.shape)
        gh = c.ptr(grad_hidden, "grad_hidden", hidden.dtype, hidden.shape)
        gt = c.ptr(grad_table, "grad_table", shape=table.shape)
        dt = _dtype_code(hidden.dtype)
        gdt = dt if grad_table is None else _dtype_code(grad_table.dtype)
        ws = c.workspace(L.zero_head_loss_workspace, n, vocab, width, dt, int(gh is not None),
                         int(gt is not None), gdt, int(piece_rows))
        loss = torch.empty(1, dtype=torch.float32, device=c.device)
        _check(L.zero_head_loss(h, t, dt, ids, size, n, vocab, width, w, int(reduction == "mean"),
                                float(grad_scale), loss.data_ptr(), ls, gh, gt, gdt,
                                int(bool(accumulate)), int(piece_rows), ws.data_ptr(), ws.numel(),
                                c.handle))
    return loss

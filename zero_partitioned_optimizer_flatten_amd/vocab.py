"""Both ends of a language model: embedding lookup and its gradient, dropout,
and softmax cross entropy against the vocabulary table. Gradients of tables go
straight into the tensor's place in a flat gradient vector.

As in the rest of the binding: checks and marshalling, the work runs in the
library's kernels on the current stream of the tensors' device (or `stream`).
Results and workspaces come from torch's allocator on that stream, so a call
can be captured in a graph.

None of the calls is an autograd function, whatever its tensors require: results
do not require gradients (embed_grad, dropout and head_loss are the backward
calls), and tensors written in place do not count it as a new version.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from typing import Optional

import torch

from . import ZERO_BF16, ZERO_F32, _check, _dtype_code, _raw_stream, _stream_handle, _torch_stream, lib

# Small calls are bound by the host: lookups that it repeats are made once.
_byref = ctypes.byref
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_DTYPES = {torch.bfloat16: ZERO_BF16, torch.float32: ZERO_F32}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
_WORDS = 1 << 64


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


class Dropout:
    """Which elements dropout drops: probability p (taken to a multiple of
    2^-16), and the counter-based generator's seed and offset, 64 bits each.
    The forward and the backward call of one place take the same; other steps
    and layers other offsets. counter: one int64 on the device, added to offset
    when the kernel runs, for steps replayed from a graph. Fixed once made."""

    __slots__ = ("_drop", "_counter")

    def __init__(self, p: float, seed: int, offset: int = 0,
                 counter: Optional[torch.Tensor] = None):
        if not (0 <= seed < _WORDS and 0 <= offset < _WORDS):
            raise ValueError("seed and offset must be in [0, 2^64)")
        at = None
        if counter is not None:
            if counter.dtype != torch.int64 or counter.numel() != 1 or counter.get_device() < 0:
                raise ValueError("counter must be one int64 on a cuda device")
            at = counter.data_ptr()
        self._counter = counter
        self._drop = _Drop(p, seed, offset, at)

    p = property(lambda self: self._drop.p)
    seed = property(lambda self: self._drop.seed)
    offset = property(lambda self: self._drop.offset)
    counter = property(lambda self: self._counter)

    def __repr__(self):
        return f"Dropout(p={self.p}, seed={self.seed}, offset={self.offset}, counter={self._counter})"


class _Call:
    """The device and stream of one call, and checks of its tensors."""

    __slots__ = ("index", "stream", "handle")

    def __init__(self, index: int, stream):
        self.index, self.stream = index, stream
        if stream is None and _raw_stream is not None:
            self.handle = _raw_stream(index)
        else:
            self.handle = _stream_handle(stream, torch.device("cuda", index))

    def ptr(self, x: torch.Tensor, what: str, dtype=None, shape=None):
        """Address of a contiguous tensor on the call's device."""
        if x.get_device() != self.index:
            raise ValueError(f"{what} is on {x.device}, the call is on cuda:{self.index}")
        if not x.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        if dtype is not None and x.dtype != dtype:
            raise TypeError(f"{what} is {x.dtype}, need {dtype}")
        if shape is not None and x.shape != shape:
            raise ValueError(f"{what} has shape {tuple(x.shape)}, need {tuple(shape)}")
        if self.stream is not None:
            x.record_stream(_torch_stream(self.stream, torch.device("cuda", self.index)))
        return x.data_ptr()

    def ids(self, x: torch.Tensor, what: str):
        """(address, bytes of an id)"""
        size = _ID_BYTES.get(x.dtype)
        if size is None:
            raise TypeError(f"{what} must be int32 or int64, got {x.dtype}")
        return self.ptr(x, what), size

    def drop(self, d: Optional[Dropout]):
        if d is None:
            return None
        if d._counter is not None:
            self.ptr(d._counter, "the dropout's counter")
        return _byref(d._drop)

    def workspace(self, like: torch.Tensor, size, *args) -> torch.Tensor:
        n = ctypes.c_int64()
        rc = size(*args, _byref(n))
        if rc:
            _check(rc)
        return like.new_empty(n.value, dtype=torch.uint8)


def _call(function):
    """The function of (call, tensor, ...) as one of (tensor, ..., stream=None):
    on the first tensor's device and the stream given, or its current one."""

    s = inspect.signature(function)
    p = list(s.parameters.values())[1:]

    @functools.wraps(function)
    def call(*args, stream=None, **kwargs):
        first = args[0] if args else kwargs.get(p[0].name)
        if first is None:
            raise TypeError(f"{function.__name__} needs {p[0].name}")
        index = first.get_device()
        if index < 0:
            raise ValueError(f"{function.__name__} runs on a cuda device, got a tensor on {first.device}")
        c = _Call(index, stream)
        if stream is None and index == _current_device():
            return function(c, *args, **kwargs)
        with torch.cuda.device(index), torch.cuda.stream(
                None if stream is None else _torch_stream(stream, torch.device("cuda", index))):
            return function(c, *args, **kwargs)

    call.__signature__ = s.replace(parameters=[
        *p, inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _code(dtype: torch.dtype) -> int:
    code = _DTYPES.get(dtype)
    return _dtype_code(dtype) if code is None else code


def _table(x: torch.Tensor, what: str):
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must have two dimensions, got {tuple(shape)}")
    return shape


@_call
def embed(call, tokens: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0,
          positions: Optional[torch.Tensor] = None, position_table: Optional[torch.Tensor] = None,
          dropout: Optional[Dropout] = None, out: Optional[torch.Tensor] = None,
          dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """dropout(scale * table[tokens] + position_table[positions]), of shape
    tokens.shape + (width,). Ids outside a table give a row of zeros. The
    result is `out`, or a new tensor of `dtype` (the table's by default)."""
    rows, width = _table(table, "table")
    if (positions is None) != (position_table is None):
        raise ValueError("positions and position_table come together")
    ids, size = call.ids(tokens, "tokens")
    at, shape = call.ptr(table, "table"), tokens.shape + (width,)
    code = _code(table.dtype)
    pos = ptable = None
    prows = 0
    if positions is not None:
        prows, pwidth = _table(position_table, "position_table")
        if pwidth != width:
            raise ValueError("table and position_table differ in width")
        pos = call.ptr(positions, "positions", tokens.dtype, tokens.shape)
        ptable = call.ptr(position_table, "position_table", table.dtype)
    if out is None:
        out = table.new_empty(shape) if dtype is None else table.new_empty(shape, dtype=dtype)
        to = out.data_ptr()
    else:
        to = call.ptr(out, "out", dtype, shape)
    rc = _lib().zero_embed(ids, size, tokens.numel(), at, rows, width, code, scale, pos, ptable,
                           prows, call.drop(dropout), to,
                           code if out.dtype == table.dtype else _code(out.dtype), call.handle)
    if rc:
        _check(rc)
    return out


@_call
def embed_grad(call, grad_out: torch.Tensor, tokens: torch.Tensor, grad_table: torch.Tensor, *,
               scale: float = 1.0, dropout: Optional[Dropout] = None,
               accumulate: bool = False) -> torch.Tensor:
    """The gradient of embed's table, written into grad_table (rows, width), a
    view of a flat gradient vector for instance, or added to the rows that
    tokens name. The gradient of its position table is embed_grad(grad_out,
    positions, grad_position_table, dropout=dropout)."""
    rows, width = _table(grad_table, "grad_table")
    n, L = tokens.numel(), _lib()
    if grad_out.numel() != n * width:
        raise ValueError(f"grad_out has {grad_out.numel()} elements, need {n * width}")
    ids, size = call.ids(tokens, "tokens")
    g, t = call.ptr(grad_out, "grad_out"), call.ptr(grad_table, "grad_table")
    gdt, tdt = _code(grad_out.dtype), _code(grad_table.dtype)
    ws = call.workspace(grad_out, L.zero_embed_grad_workspace, n, rows, width)
    rc = L.zero_embed_grad(g, gdt, ids, size, n, rows, width, scale, call.drop(dropout), t, tdt,
                           bool(accumulate), ws.data_ptr(), ws.numel(), call.handle)
    if rc:
        _check(rc)
    return grad_table


@_call
def dropout(call, x: torch.Tensor, drop: Dropout, *, add: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dropout(x), plus `add` if given; dropout(grad, drop) is its backward.
    out may be x or add."""
    at = call.ptr(x, "x")
    code = _code(x.dtype)
    residual = None if add is None else call.ptr(add, "add", x.dtype, x.shape)
    if out is None:
        out = torch.empty_like(x)
        to = out.data_ptr()
    else:
        to = call.ptr(out, "out", x.dtype, x.shape)
    rc = _lib().zero_dropout(at, residual, to, x.numel(), code, call.drop(drop), call.handle)
    if rc:
        _check(rc)
    return out


@_call
def head_loss(call, hidden: torch.Tensor, table: torch.Tensor, targets: torch.Tensor, *,
              weights: Optional[torch.Tensor] = None, reduction: str = "mean",
              grad_scale: float = 1.0, losses: Optional[torch.Tensor] = None,
              grad_hidden: Optional[torch.Tensor] = None,
              grad_table: Optional[torch.Tensor] = None, accumulate: bool = False,
              piece_rows: int = 0) -> torch.Tensor:
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
    L, n, shape = _lib(), targets.numel(), targets.shape
    if hidden.shape != shape + (width,):
        raise ValueError(f"hidden has shape {tuple(hidden.shape)}, need {(*shape, width)}")
    ids, size = call.ids(targets, "targets")
    h, t = call.ptr(hidden, "hidden"), call.ptr(table, "table", hidden.dtype)
    dt = _code(hidden.dtype)
    w = None if weights is None else call.ptr(weights, "weights", torch.float32, shape)
    ls = None if losses is None else call.ptr(losses, "losses", torch.float32, shape)
    gh = None if grad_hidden is None else call.ptr(grad_hidden, "grad_hidden", hidden.dtype, hidden.shape)
    gt, gdt = None, dt
    if grad_table is not None:
        gt, gdt = call.ptr(grad_table, "grad_table", None, table.shape), _code(grad_table.dtype)
    ws = call.workspace(hidden, L.zero_head_loss_workspace, n, vocab, width, dt, gh is not None,
                        gt is not None, gdt, piece_rows)
    loss = hidden.new_empty(1, dtype=torch.float32)
    rc = L.zero_head_loss(h, t, dt, ids, size, n, vocab, width, w, reduction == "mean", grad_scale,
                          loss.data_ptr(), ls, gh, gt, gdt, bool(accumulate), piece_rows,
                          ws.data_ptr(), ws.numel(), call.handle)
    if rc:
        _check(rc)
    return loss

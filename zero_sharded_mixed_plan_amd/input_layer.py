"""The model's input layer over torch device tensors: embedding lookup, its
gradient, and dropout from a counter-based generator.

The tables are tensors of the all-gather buffer that the sharded step writes
(ZeroAdam.param), the gradients tensors of a flat gradient buffer that it reads
(ZeroAdam.grad_view).  torch supplies device memory and the stream (the current
stream of the tensors' device); every step of the computation runs in
libzero_shard.so (zero_embed_lookup, zero_embed_grad, zero_dropout).

The calls record no history for autograd: a loop calls the backward pass itself, or
from a torch.autograd.Function.  With grad mode on, a tensor that requires grad is
refused, since its gradient would be lost without a sign; detach it, or call under
torch.no_grad() (inside a Function's forward and backward, grad mode is off).
"""
from __future__ import annotations

import ctypes
import struct
from typing import Callable, Optional, Union

import torch

from . import _abi
from .optim import _CODES, dtype_code

_ID_BYTES = {torch.int32: 4, torch.int64: 8}

# The calls' host time is what the smallest sizes cost, so the argument structs are
# packed in one go (native layout, as the header declares them; the sizes are
# checked against the ctypes declarations below) and the stream is asked for by number.
_EMBED = struct.Struct("@PqqqiiPqqfPqqPqPqiP")
_GRAD = struct.Struct("@PqiiPqqqqqfiPqiPPq")
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
assert _EMBED.size == ctypes.sizeof(_abi.zero_embed_args_t)
assert _GRAD.size == ctypes.sizeof(_abi.zero_embed_grad_args_t)


class Dropout:
    """One dropout of one step (zero_drop_t): which elements of a [rows, cols]
    matrix are dropped is a function of seed, site, step, the row's place in the
    whole batch (row0 + row) and the column.

    step: an integer; a function that gives one, asked at every call; or a device
    int64 tensor of one element that the kernels read when they run (a captured
    graph then draws a new mask at every replay).  ZeroAdam.dropout passes the count
    of the steps applied in one of the last two forms.  The tensor must stay alive
    until the work is done.
    """
    __slots__ = ("c", "_step", "_count", "_ref")

    def __init__(self, p: float, seed: int = 0, site: int = 0,
                 step: Union[int, Callable[[], int], torch.Tensor] = 0, row0: int = 0):
        self._step = self._count = None
        if callable(step):
            self._count = step
            step = step()
        if isinstance(step, torch.Tensor):
            if step.dtype != torch.int64 or step.numel() != 1 or not step.is_cuda:
                raise ValueError("step must be an integer or a device int64 tensor of one element")
            self._step = step
            step = 0
        if not (0 <= site < 1 << 32 and 0 <= step < 1 << 32 and 0 <= row0 < 1 << 32):
            raise ValueError("site, row0 or step out of range")
        self.c = c = _abi.zero_drop_t(p, seed & 0xFFFFFFFFFFFFFFFF, site, 0, step,
                                      None if self._step is None else self._step.data_ptr(), row0)
        self._ref = ctypes.addressof(c)

    @property
    def p(self) -> float:
        return self.c.p


def _device(first: torch.Tensor, *others) -> int:
    """The index of the tensors' one GPU."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors are on different devices" if t.is_cuda else "tensors must be on the GPU")
    return dev


def _no_history() -> None:
    """Called where a tensor requires grad."""
    if torch.is_grad_enabled():
        raise ValueError("a tensor requires grad, and these calls record no history for autograd: "
                         "detach it, or call under torch.no_grad()")


def _call(fn, dev, *args):
    """Run a library call on the current stream of device `dev`, with it current."""
    if dev == _current_device():
        rc = fn(*args, _current_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _current_stream(dev))
    if rc != _abi.ZERO_OK:
        _abi._check(rc)


def _rows(t: torch.Tensor, what: str):
    """A tensor [..., cols] as rows: (rows, cols, stride between rows)."""
    shape = t.shape
    if t.is_contiguous():
        if len(shape) == 2:
            return shape[0], shape[1], shape[1]
        if len(shape) == 0:
            raise ValueError(f"{what}: a tensor without dimensions has no rows")
        n = 1
        for s in shape[:-1]:
            n *= s
        return n, shape[-1], shape[-1]
    if len(shape) != 2:
        raise ValueError(f"{what}: a tensor that is not a matrix must be contiguous")
    n, c = shape
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the columns must be adjacent")
    ld = t.stride(0) if n > 1 else c
    if ld < c:
        raise ValueError(f"{what}: the rows must not overlap")
    return n, c, ld


def _code(dt: torch.dtype) -> int:
    return _CODES[dt] if dt in _CODES else dtype_code(dt)


def _flat_ids(t: torch.Tensor, what: str) -> int:
    try:
        b = _ID_BYTES[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be int32 or int64, not {t.dtype}") from None
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return b


def _drop(drop: Optional[Dropout], dev: int) -> int:
    if drop is None:
        return 0
    if drop._step is not None and drop._step.device.index != dev:
        raise ValueError("the dropout's step is on another device")
    if drop._count is not None:
        drop.c.step = drop._count()
    return drop._ref


def dropout(x: torch.Tensor, drop: Optional[Dropout], *, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Kept elements of x times 1 / (1 - p), dropped ones 0, plus `residual`.

    x [..., cols] is a matrix of rows and columns to the generator.  The result has
    x's shape and, in this order, the type of out, out_dtype, the residual, x.
    out may be x or residual.  The backward pass is dropout(dout, drop, out_dtype=x.dtype).
    """
    n, cols, ld_x = _rows(x, "x")
    given = out
    if out is None:
        dt = out_dtype or (x if residual is None else residual).dtype
        out = torch.empty_like(x) if dt is x.dtype and ld_x == cols else x.new_empty(x.shape, dtype=dt)
        ld_out = cols
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out has another type than out_dtype")
        if out.shape != x.shape:
            raise ValueError("x, residual and out must have one shape")
        ld_out = _rows(out, "out")[2]
    ptr_r = ld_r = 0
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("x, residual and out must have one shape")
        if residual.dtype != out.dtype:
            raise ValueError("residual and out must have one type")
        ptr_r, ld_r = residual.data_ptr(), _rows(residual, "residual")[2]
    if (x.requires_grad or residual is not None and residual.requires_grad
            or given is not None and given.requires_grad):
        _no_history()
    dev = _device(x, residual, given)
    if n == 0 or cols == 0:
        return out
    _call(_abi.lib().zero_dropout, dev, x.data_ptr(), ld_x, _code(x.dtype), ptr_r, ld_r, out.data_ptr(), ld_out,
          _code(out.dtype), n, cols, _drop(drop, dev))
    return out


def embedding(ids: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0, id0: int = 0,
              pos_table: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None, pos_period: int = 0,
              drop: Optional[Dropout] = None, out: Optional[torch.Tensor] = None,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """dropout(scale * table[ids - id0] + pos_table[pos]), [*ids.shape, dim].

    table [rows, dim] holds the ids id0 .. id0 + rows - 1; an id outside reads a row
    of zeros.  pos: one position per id, or None for t % pos_period with t the
    id's place in ids.  The dropout's row is t.
    """
    if table.dim() != 2:
        raise ValueError("table must be a matrix")
    idb = _flat_ids(ids, "ids")
    rows, dim, ld = _rows(table, "table")
    given = out
    if out is None:
        out = table.new_empty((*ids.shape, dim), dtype=out_dtype or table.dtype)
        ld_out = dim
    elif out.shape != (*ids.shape, dim) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [*ids.shape, dim] of out_dtype")
    else:
        ld_out = _rows(out, "out")[2]
    ptr_pt = ld_pt = n_pt = ptr_pos = 0
    if pos_table is not None:
        n_pt, pos_dim, ld_pt = _rows(pos_table, "pos_table")
        if pos_table.dim() != 2 or pos_dim != dim or pos_table.dtype != table.dtype:
            raise ValueError("pos_table must be [positions, dim] of the table's type")
        ptr_pt = pos_table.data_ptr()
        if pos is not None:
            if pos.shape != ids.shape or pos.dtype != ids.dtype:
                raise ValueError("pos must have the shape and type of ids")
            _flat_ids(pos, "pos")
            if n_pt:  # a table without rows has no address: its positions all read zeros
                ptr_pos = pos.data_ptr()
        elif pos_period < 1:
            raise ValueError("pos_table needs pos or a pos_period of at least 1")
    elif pos is not None:
        raise ValueError("pos without a pos_table")
    if (table.requires_grad or pos_table is not None and pos_table.requires_grad
            or given is not None and given.requires_grad):
        _no_history()
    dev = _device(table, ids, given, pos_table, pos)
    n = ids.numel()
    if n == 0 or dim == 0:
        return out
    _call(_abi.lib().zero_embed_lookup, dev, _EMBED.pack(
        table.data_ptr(), ld, rows, id0, _code(table.dtype), idb, ids.data_ptr(), n, dim, scale,
        ptr_pt, ld_pt, n_pt, ptr_pos, pos_period, out.data_ptr(), ld_out, _code(out.dtype),
        _drop(drop, dev)))
    return out


def embedding_grad_workspace(n_ids: int, rows: int, dim: int, device="cuda") -> torch.Tensor:
    """A workspace for embedding_grad calls of at most these sizes that do not
    overlap in time."""
    n = _abi.lib().zero_embed_grad_ws_bytes(n_ids, rows, dim)
    if n == 0:
        raise ValueError("sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=device)


def embedding_grad(dy: torch.Tensor, ids: Optional[torch.Tensor], grad: torch.Tensor, *, scale: float = 1.0,
                   id0: int = 0, period: int = 0, drop: Optional[Dropout] = None, accumulate: bool = False,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """grad[v] = scale * sum of dropout'(dy[t]) over ids[t] == id0 + v, written to
    every row of grad [rows, dim], or added to what it holds (accumulate).

    ids None: the id of row t of dy is t % period (a table of positions).  drop:
    the lookup's.  workspace: see embedding_grad_workspace (None: allocated here).
    Returns grad.
    """
    if grad.dim() != 2:
        raise ValueError("grad must be a matrix")
    rows, dim, ld_grad = _rows(grad, "grad")
    n, cols, ld_dy = _rows(dy, "dy")
    if cols != dim:
        raise ValueError("dy and grad must have one width")
    ptr_ids, idb = 0, 8
    if ids is not None:
        if ids.shape != dy.shape[:-1]:
            raise ValueError("dy must be [*ids.shape, dim]")
        idb = _flat_ids(ids, "ids")
        ptr_ids = ids.data_ptr() if n else 0
    elif period < 1:
        raise ValueError("ids None needs a period of at least 1")
    if dy.requires_grad or grad.requires_grad:
        _no_history()
    dev = _device(grad, dy, ids, workspace)
    if rows == 0 or dim == 0:
        return grad
    L = _abi.lib()
    if workspace is None:
        workspace = grad.new_empty(L.zero_embed_grad_ws_bytes(n, rows, dim), dtype=torch.uint8)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    _call(L.zero_embed_grad, dev, _GRAD.pack(
        dy.data_ptr(), ld_dy, _code(dy.dtype), idb, ptr_ids, max(period, 1), n, dim, id0, rows, scale,
        _code(grad.dtype), grad.data_ptr(), ld_grad, 1 if accumulate else 0, _drop(drop, dev),
        workspace.data_ptr(), workspace.numel()))
    return grad

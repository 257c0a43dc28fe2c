"""The model's input layer over torch device tensors: embedding lookup, its
gradient, and dropout from a counter-based generator.

The tables are tensors of the all-gather buffer that the sharded step writes
(ZeroAdam.param), the gradients tensors of a flat gradient buffer that it reads
(ZeroAdam.grad_view).  torch supplies device memory and the stream (the current
stream of the tensors' device); every step of the computation runs in
libzero_shard.so (zero_embed_lookup, zero_embed_grad, zero_dropout).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Union

import torch

from . import _abi
from .optim import dtype_code

_ID_BYTES = {torch.int32: 4, torch.int64: 8}


class Dropout:
    """One dropout of one step (zero_drop_t): which elements of a [rows, cols]
    matrix are dropped is a function of seed, site, step, the row's place in the
    whole batch (row0 + row) and the column.

    step: an integer, or a device int64 tensor of one element that the kernels
    read when they run (a captured graph then draws a new mask at every replay;
    ZeroAdam.dropout passes the step control's count).  The tensor must stay alive
    until the work is done.
    """
    __slots__ = ("c", "_step", "_ref")

    def __init__(self, p: float, seed: int = 0, site: int = 0, step: Union[int, torch.Tensor] = 0, row0: int = 0):
        c = _abi.zero_drop_t()
        c.p = p
        c.seed = seed & 0xFFFFFFFFFFFFFFFF
        c.site = site
        c.row0 = row0
        self._step = None
        if isinstance(step, torch.Tensor):
            if step.dtype != torch.int64 or step.numel() != 1 or not step.is_cuda:
                raise ValueError("step must be an integer or a device int64 tensor of one element")
            self._step = step
            c.step_dev = step.data_ptr()
        else:
            c.step = step
        if c.site != site or c.row0 != row0 or (self._step is None and c.step != step):
            raise ValueError("site, row0 or step out of range")
        self.c = c
        self._ref = ctypes.addressof(c)

    @property
    def p(self) -> float:
        return self.c.p


def _place(*tensors):
    """The one device of the tensors; its current stream."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on the GPU")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors are on different devices")
    return dev, torch.cuda.current_stream(dev).cuda_stream


def _call(fn, dev, *args):
    """Run a library call with the tensors' device current."""
    if dev.index == torch.cuda.current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != _abi.ZERO_OK:
        _abi._check(rc)


def _rows(t: torch.Tensor, what: str):
    """A tensor [..., cols] as rows: (rows, cols, stride between rows)."""
    if t.dim() == 2:
        n, c = t.shape
        if n <= 1 or t.is_contiguous():
            if c > 1 and t.stride(1) != 1:
                raise ValueError(f"{what}: the columns must be adjacent")
            return n, c, c
        if (c > 1 and t.stride(1) != 1) or t.stride(0) < c:
            raise ValueError(f"{what}: the columns must be adjacent and the rows apart")
        return n, c, t.stride(0)
    if t.dim() == 0 or not t.is_contiguous():
        raise ValueError(f"{what}: a tensor that is not a matrix must be contiguous")
    c = t.shape[-1]
    n = 1
    for s in t.shape[:-1]:
        n *= s
    return n, c, c


def _flat_ids(t: torch.Tensor, what: str) -> int:
    try:
        b = _ID_BYTES[t.dtype]
    except KeyError:
        raise TypeError(f"{what} must be int32 or int64, not {t.dtype}") from None
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return b


def _drop(drop: Optional[Dropout], dev):
    if drop is None:
        return None
    if drop._step is not None and drop._step.device != dev:
        raise ValueError("the dropout's step is on another device")
    return drop._ref


def dropout(x: torch.Tensor, drop: Optional[Dropout], *, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Kept elements of x times 1 / (1 - p), dropped ones 0, plus `residual`.

    x [..., cols] is a matrix of rows and columns to the generator.  The result has
    x's shape and, in this order, the type of out, out_dtype, the residual, x.
    out may be x or residual.  The backward pass is dropout(dout, drop, out_dtype=x.dtype).
    """
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype or (x if residual is None else residual).dtype, device=x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out has another type than out_dtype")
    if out.shape != x.shape or (residual is not None and residual.shape != x.shape):
        raise ValueError("x, residual and out must have one shape")
    if residual is not None and residual.dtype != out.dtype:
        raise ValueError("residual and out must have one type")
    dev, st = _place(x, residual, out)
    n, cols, ld_x = _rows(x, "x")
    if n == 0 or cols == 0:
        return out
    ld_r = 0 if residual is None else _rows(residual, "residual")[2]
    _call(_abi.lib().zero_dropout, dev, x.data_ptr(), ld_x, dtype_code(x.dtype),
          None if residual is None else residual.data_ptr(), ld_r, out.data_ptr(), _rows(out, "out")[2],
          dtype_code(out.dtype), n, cols, _drop(drop, dev), st or None)
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
    if out is None:
        out = torch.empty((*ids.shape, dim), dtype=out_dtype or table.dtype, device=table.device)
    elif out.shape != (*ids.shape, dim) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out must be [*ids.shape, dim] of out_dtype")
    a = _abi.zero_embed_args_t()
    if pos_table is not None:
        if pos_table.dim() != 2 or pos_table.shape[1] != dim or pos_table.dtype != table.dtype:
            raise ValueError("pos_table must be [positions, dim] of the table's type")
        a.pos_rows, _, a.ld_pos = _rows(pos_table, "pos_table")
        a.pos_table = pos_table.data_ptr()
        if pos is not None:
            if pos.shape != ids.shape or pos.dtype != ids.dtype:
                raise ValueError("pos must have the shape and type of ids")
            _flat_ids(pos, "pos")
            a.pos = pos.data_ptr()
        elif pos_period < 1:
            raise ValueError("pos_table needs pos or a pos_period of at least 1")
        a.pos_period = pos_period
    elif pos is not None:
        raise ValueError("pos without a pos_table")
    dev, st = _place(ids, table, out, pos_table, pos)
    n = ids.numel()
    if n == 0 or dim == 0:
        return out
    a.table = table.data_ptr()
    a.ld_table = ld
    a.rows = rows
    a.id0 = id0
    a.table_dtype = dtype_code(table.dtype)
    a.id_bytes = idb
    a.ids = ids.data_ptr()
    a.n_ids = n
    a.dim = dim
    a.scale = scale
    a.out = out.data_ptr()
    a.ld_out = _rows(out, "out")[2]
    a.out_dtype = dtype_code(out.dtype)
    a.drop = _drop(drop, dev)
    _call(_abi.lib().zero_embed_lookup, dev, ctypes.addressof(a), st or None)
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
    a = _abi.zero_embed_grad_args_t()
    a.id_bytes = 8
    if ids is not None:
        if ids.shape != dy.shape[:-1]:
            raise ValueError("dy must be [*ids.shape, dim]")
        a.id_bytes = _flat_ids(ids, "ids")
        a.ids = ids.data_ptr() if n else None
    elif period < 1:
        raise ValueError("ids None needs a period of at least 1")
    a.period = max(period, 1)
    dev, st = _place(dy, grad, ids, workspace)
    if rows == 0 or dim == 0:
        return grad
    L = _abi.lib()
    if workspace is None:
        need = L.zero_embed_grad_ws_bytes(n, rows, dim)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    a.dy = dy.data_ptr()
    a.ld_dy = ld_dy
    a.dy_dtype = dtype_code(dy.dtype)
    a.n_ids = n
    a.dim = dim
    a.id0 = id0
    a.rows = rows
    a.scale = scale
    a.grad_dtype = dtype_code(grad.dtype)
    a.grad = grad.data_ptr()
    a.ld_grad = ld_grad
    a.accumulate = 1 if accumulate else 0
    a.drop = _drop(drop, dev)
    a.ws = workspace.data_ptr()
    a.ws_bytes = workspace.numel()
    _call(L.zero_embed_grad, dev, ctypes.addressof(a), st or None)
    return grad

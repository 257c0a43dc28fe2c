"""The pre-norm gated feed-forward sub-layer over torch device tensors: RMS norm with
the residual's addition, activation checkpoints in 8 bits, the gated projections, and
the backward passes of all of them.

The weights are tensors of the all-gather buffer that the sharded step writes
(ZeroAdam.param), their gradients tensors of a flat gradient buffer that it reads
(ZeroAdam.grad_view).  torch supplies device memory and the stream (the current
stream of the tensors' device); every step of the computation runs in libzero_shard.so
(zero_rms_norm, zero_pack8, zero_gated, ...).

    n = rms_norm(x, w_norm, eps=1e-5, residual=stream, packed=True)
    f = gated(n.y, w_gate, w_up, keep="packed")
    ...                                               # f.a through the down projection
    g = gated_grad(da, f.gate, f.up, again=True)      # g.a for the down projection's gradient
    dn = gated_input_grad(g.gate, g.up, w_gate, w_up)
    gated_weight_grad(g.gate, g.up, unpack8(n.packed, dtype), grad_gate, grad_up)
    dh = rms_norm_grad(dn, n.total, n.rstd, w_norm, residual_grad=d, weight_grad=grad_norm)

Matrices [..., cols] are rows of the last dimension; one that is not contiguous has to
have two dimensions and adjacent columns.  Inputs and results may be column ranges of one buffer.  The calls record no history for autograd: a loop
calls the backward pass itself, or from a torch.autograd.Function.  With grad mode on, a
tensor that requires grad is refused, since its gradient would be lost without a sign, and so is
one that carries a tangent of forward-mode differentiation.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import _abi
from .input_layer import _call, _code, _forward_ad, _no_history, _no_tangents, _rows

# as in input_layer: the calls' argument structs are packed in one go
_RMS = struct.Struct("@PqiiPqPqPiiPqPPqqd")
_RMS_GRAD = struct.Struct("@PqiiPqPPPiiPqPqPiiqqPq")
_GATED = struct.Struct("@qqqii" + "Pq" * 6 + "PP" + "Pq" * 6 + "iiPq")
_ZEROS = tuple((0,) * n for n in range(17))  # what a call leaves out
assert _RMS.size == ctypes.sizeof(_abi.zero_rms_args_t)
assert _RMS_GRAD.size == ctypes.sizeof(_abi.zero_rms_grad_args_t)
assert _GATED.size == ctypes.sizeof(_abi.zero_gated_args_t)

BLOCK = 32  # columns that share a scale
_ACTS = {"silu": 0, "gelu": 1}


class Packed8(NamedTuple):
    """A matrix [..., cols] held in 8 bits: codes [..., cols] (float8_e4m3fn, or uint8)
    and scales [..., ceil(cols / 32)] (float8_e8m0fnu, or uint8).  What it stands for
    is codes times the scale of their 32 columns."""
    codes: torch.Tensor
    scales: torch.Tensor


class Normed(NamedTuple):
    y: Optional[torch.Tensor]
    packed: Optional[Packed8]
    total: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


class Gated(NamedTuple):
    a: torch.Tensor
    gate: Union[torch.Tensor, Packed8, None]
    up: Union[torch.Tensor, Packed8, None]


class GatedGrad(NamedTuple):
    gate: torch.Tensor
    up: torch.Tensor
    a: Optional[torch.Tensor]


_CODE_TYPES = (torch.float8_e4m3fn, torch.uint8)
_SCALE_TYPES = (torch.float8_e8m0fnu, torch.uint8)


def packed8_empty(shape, device="cuda") -> Packed8:
    """Memory for a matrix of this shape held in 8 bits."""
    *lead, cols = shape
    codes = torch.empty((*lead, cols), dtype=torch.float8_e4m3fn, device=device)
    return Packed8(codes, torch.empty((*lead, (cols + BLOCK - 1) // BLOCK), dtype=torch.float8_e8m0fnu, device=device))


def _packed8(shape, like: torch.Tensor) -> Packed8:
    """packed8_empty beside a tensor."""
    if like.shape == shape:  # a quicker call
        codes = torch.empty_like(like, dtype=torch.float8_e4m3fn, memory_format=torch.contiguous_format)
    else:
        codes = like.new_empty(shape, dtype=torch.float8_e4m3fn)
    return Packed8(codes, like.new_empty((*shape[:-1], (shape[-1] + BLOCK - 1) // BLOCK), dtype=torch.float8_e8m0fnu))


def _held(p: Packed8, rows: int, cols: int, shape, what: str) -> _abi.zero_held_t:
    """The C struct of a Packed8 of this shape."""
    codes, scales = p.codes, p.scales
    if codes.dtype not in _CODE_TYPES or scales.dtype not in _SCALE_TYPES:
        raise TypeError(f"{what}: codes must be float8_e4m3fn or uint8, scales float8_e8m0fnu or uint8")
    if codes.shape != shape or scales.shape != (*shape[:-1], (cols + BLOCK - 1) // BLOCK):
        raise ValueError(f"{what}: codes must be {list(shape)}, scales one for each {BLOCK} columns")
    ld_codes = _rows(codes, what)[2]
    ld_scales = _rows(scales, what)[2]
    if rows == 0:
        return _abi.zero_held_t()
    return _abi.zero_held_t(codes.data_ptr(), ld_codes, scales.data_ptr(), ld_scales)


def _is_packed(t) -> bool:
    return isinstance(t, Packed8)


def _one_device(first: torch.Tensor, *others) -> int:
    """The index of the one GPU of what a caller gave: tensors, Packed8s and Nones."""
    if _forward_ad._current_level >= 0:
        _no_tangents(first, *others)
    dev = first.get_device()
    history, stranger = first.requires_grad, None
    for t in others:
        if t is None or t is True or t is False:
            continue
        if isinstance(t, Packed8):
            _one_device(first, *t)
            continue
        if t.get_device() != dev:
            stranger = t
        history = history or t.requires_grad
    if history:
        _no_history()
    if dev < 0 or (stranger is not None and not stranger.is_cuda):
        raise ValueError("tensors must be on the GPU")
    if stranger is not None:
        raise ValueError("tensors are on different devices")
    return dev


def _result(out: Optional[torch.Tensor], shape, dtype: torch.dtype, like: torch.Tensor, what: str):
    """A given result, checked, or a new one: (tensor, stride between rows)."""
    if out is None:
        if like.shape == shape:  # a quicker call
            return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format), shape[-1]
        return like.new_empty(shape, dtype=dtype), shape[-1]
    if out.shape != shape or out.dtype != dtype:
        raise ValueError(f"{what} must be {list(shape)} of {dtype}")
    return out, _rows(out, what)[2]


def _vector(t: torch.Tensor, n: int, what: str) -> None:
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} elements")


# ---------------------------------------------------------------------------
# 8 bits
# ---------------------------------------------------------------------------

def pack8(x: torch.Tensor, *, out: Optional[Packed8] = None) -> Packed8:
    """x [..., cols] held in 8 bits: a checkpoint of about a byte an element."""
    n, cols, ld = _rows(x, "x")
    code = _code(x.dtype)
    p = _packed8(x.shape, x) if out is None else out
    held = _held(p, n, cols, x.shape, "out")
    dev = _one_device(x, out)
    if n and cols:
        _call(_abi.lib().zero_pack8, dev, x.data_ptr(), ld, code, n, cols, ctypes.addressof(held))
    return p


def unpack8(p: Packed8, dtype: Optional[torch.dtype] = None, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that p stands for, exact in bf16 and fp32 down to their smallest numbers, in fp16 within its range
    (dtype: default out's, or bf16)."""
    dtype = dtype or (torch.bfloat16 if out is None else out.dtype)
    code = _code(dtype)
    n, cols, _ = _rows(p.codes, "codes")
    held = _held(p, n, cols, p.codes.shape, "p")
    given = out
    out, ld = _result(out, p.codes.shape, dtype, p.codes, "out")
    dev = _one_device(p.codes, p.scales, given)
    if n and cols:
        _call(_abi.lib().zero_unpack8, dev, ctypes.addressof(held), n, cols, out.data_ptr(), ld, code)
    return out


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *, eps: float,
             residual: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
             out: Union[torch.Tensor, bool] = True, out_dtype: Optional[torch.dtype] = None,
             packed: Union[Packed8, bool] = False, rstd: Union[torch.Tensor, bool] = True) -> Normed:
    """y = h * rstd * weight with h = x + residual and rstd = 1 / sqrt(mean(h^2) + eps).

    x [..., cols], 1 to 8192 columns; residual of x's type or fp32; total receives h in the residual's
    type (a new tensor, or one given, which may be the residual or x itself).  y has, in this
    order, the type of out, out_dtype, x; out=False leaves it out.  packed: y in 8
    bits too, or only.  rstd: fp32, [...]; False leaves it out.
    """
    n, cols, ld_x = _rows(x, "x")
    if cols == 0:
        raise ValueError("x has no columns")
    shape = x.shape
    xc = _code(x.dtype)
    ptr_r = ld_r = ptr_t = ld_t = 0
    given_total = None
    rc = xc
    if residual is not None:
        if residual.shape != shape:
            raise ValueError("x and residual must have one shape")
        rc = _code(residual.dtype)
        ld_r = _rows(residual, "residual")[2]
        given_total = total
        total, ld_t = _result(total, shape, residual.dtype, x, "total")
        ptr_r, ptr_t = residual.data_ptr(), total.data_ptr()
    elif total is not None:
        raise ValueError("total without a residual")
    ptr_w = wc = 0
    if weight is not None:
        _vector(weight, cols, "weight")
        ptr_w, wc = weight.data_ptr(), _code(weight.dtype)
    y, ptr_y, ld_y, yc = None, 0, 0, 0
    if out is not False:
        given = None if out is True else out
        dt = out_dtype or (x if given is None else given).dtype
        y, ld_y = _result(given, shape, dt, x, "out")
        ptr_y, yc = y.data_ptr(), _code(dt)
    held = keep = None
    if packed is not False:
        keep = _packed8(shape, x) if packed is True else packed
        held = _held(keep, n, cols, shape, "packed")
    if y is None and keep is None:
        raise ValueError("neither out nor packed is asked for")
    scale = None
    if rstd is True:
        scale = x.new_empty(shape[:-1], dtype=torch.float32)
    elif rstd is not False:
        scale = rstd
        if scale.shape != shape[:-1] or scale.dtype != torch.float32 or not scale.is_contiguous():
            raise ValueError("rstd must be contiguous fp32 of x's shape without the columns")
    dev = _one_device(x, residual, weight, given_total, out, packed, rstd)
    if n:
        _call(_abi.lib().zero_rms_norm, dev, _RMS.pack(
            x.data_ptr(), ld_x, xc, rc, ptr_r, ld_r, ptr_t, ld_t, ptr_w, wc, yc, ptr_y, ld_y,
            0 if held is None else ctypes.addressof(held), 0 if scale is None else scale.data_ptr(), n, cols, eps))
    return Normed(y, keep, total, scale)


def rms_norm_grad_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A workspace for rms_norm_grad calls of at most these sizes that do not overlap in time."""
    n = _abi.lib().zero_rms_grad_ws_bytes(rows, cols)
    if n == 0:
        raise ValueError("sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, like: torch.Tensor) -> torch.Tensor:
    if workspace is None:
        return like.new_empty(nbytes, dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")
    return workspace


def rms_norm_grad(dy: torch.Tensor, h: Union[torch.Tensor, Packed8], rstd: torch.Tensor,
                  weight: Optional[torch.Tensor] = None, *, residual_grad: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                  weight_grad: Optional[torch.Tensor] = None, accumulate: bool = False,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of rms_norm in h, plus residual_grad (the gradient that reaches h past
    the norm), and in the weight, written to weight_grad or added to what it holds (accumulate).

    dy [..., cols], 1 to 8192 columns.  h: what the norm was taken of (x, or total), as it
    was or from pack8.  rstd: the forward pass's, finite (it is infinite for rows below
    2^-128 without an eps).  The result has the type of, in this order, h as a tensor, out,
    out_dtype, residual_grad, dy: dy's type or fp32.  out may be dy, h or residual_grad.
    """
    n, cols, ld_dy = _rows(dy, "dy")
    shape = dy.shape
    if _is_packed(h):
        given = out if out is not None else residual_grad if out_dtype is None else None
        dt = out_dtype or dy.dtype if given is None else given.dtype
        held = _held(h, n, cols, shape, "h")
        ptr_h = ld_h = 0
    else:
        if h.shape != shape:
            raise ValueError("dy and h must have one shape")
        held, dt = None, h.dtype
        ptr_h, ld_h = h.data_ptr(), _rows(h, "h")[2]
    if out_dtype is not None and out_dtype != dt:
        raise ValueError("out_dtype is another type than h's or out's")
    yc, hc = _code(dy.dtype), _code(dt)
    if rstd.shape != shape[:-1] or rstd.dtype != torch.float32 or not rstd.is_contiguous():
        raise ValueError("rstd must be contiguous fp32 of dy's shape without the columns")
    ptr_w = wc = ptr_d = ld_d = ptr_dw = dwc = 0
    if weight is not None:
        _vector(weight, cols, "weight")
        ptr_w, wc = weight.data_ptr(), _code(weight.dtype)
    if residual_grad is not None:
        if residual_grad.shape != shape or residual_grad.dtype != dt:
            raise ValueError(f"residual_grad must be {list(shape)} of {dt}")
        ptr_d, ld_d = residual_grad.data_ptr(), _rows(residual_grad, "residual_grad")[2]
    if weight_grad is not None:
        _vector(weight_grad, cols, "weight_grad")
        ptr_dw, dwc = weight_grad.data_ptr(), _code(weight_grad.dtype)
    elif accumulate:
        raise ValueError("accumulate without a weight_grad")
    given = out
    out, ld_out = _result(out, shape, dt, dy, "out")
    dev = _one_device(dy, h, rstd, weight, residual_grad, given, weight_grad, workspace)
    if cols == 0 or (n == 0 and weight_grad is None):
        return out
    L = _abi.lib()
    ptr_ws = n_ws = 0
    if weight_grad is not None:
        workspace = _workspace(workspace, L.zero_rms_grad_ws_bytes(n, cols), dy)
        ptr_ws, n_ws = workspace.data_ptr(), workspace.numel()
    _call(L.zero_rms_norm_grad, dev, _RMS_GRAD.pack(
        dy.data_ptr(), ld_dy, yc, hc, ptr_h, ld_h, 0 if held is None else ctypes.addressof(held), rstd.data_ptr(),
        ptr_w, wc, dwc, ptr_d, ld_d, out.data_ptr(), ld_out, ptr_dw, 1 if accumulate else 0, 0, n, cols, ptr_ws, n_ws))
    return out


# ---------------------------------------------------------------------------
# the gated block
# ---------------------------------------------------------------------------

def _act(act: str) -> int:
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, not {act!r}") from None


def _kept(gate, up, n: int, hidden: int, shape, like: torch.Tensor):
    """The arguments g, ld_g, u, ld_u, g8, u8 of a pair of tensors or Packed8s, or of none, and what
    holds the structs."""
    if gate is None or up is None:
        if gate is not up:
            raise ValueError("gate and up go together: both or neither")
        return 0, 0, 0, 0, 0, 0, None
    if isinstance(gate, Packed8) != isinstance(up, Packed8):
        raise ValueError("gate and up must be of one form")
    if isinstance(gate, Packed8):
        held = _held(gate, n, hidden, shape, "gate"), _held(up, n, hidden, shape, "up")
        return 0, 0, 0, 0, ctypes.addressof(held[0]), ctypes.addressof(held[1]), held
    for t, what in ((gate, "gate"), (up, "up")):
        if t.shape != shape or t.dtype != like.dtype:
            raise ValueError(f"{what} must be {list(shape)} of {like.dtype}")
    return gate.data_ptr(), _rows(gate, "gate")[2], up.data_ptr(), _rows(up, "up")[2], 0, 0, None


def _weights(w_gate: torch.Tensor, w_up: torch.Tensor, dtype: torch.dtype):
    shape = w_gate.shape
    if len(shape) != 2 or shape != w_up.shape or w_gate.dtype != dtype or w_up.dtype != dtype:
        raise ValueError(f"w_gate and w_up must be [hidden, dim] of {dtype}")
    return shape[0], shape[1], _rows(w_gate, "w_gate")[2], _rows(w_up, "w_up")[2]


def gated(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *, act: str = "silu",
          out: Optional[torch.Tensor] = None,
          keep: Union[None, str, Tuple[torch.Tensor, torch.Tensor], Tuple[Packed8, Packed8]] = None) -> Gated:
    """a = act(x w_gate^T) * (x w_up^T), [..., hidden], in one kernel.

    x [..., dim], weights [hidden, dim], all of one type.  act: "silu", or "gelu" in its
    tanh form.  keep: gate and up for the backward pass, in new tensors of x's type ("tensors") or
    in 8 bits ("packed"), or a pair of either to write to.
    """
    n, dim, ld_x = _rows(x, "x")
    kind, code = _act(act), _code(x.dtype)
    hidden, wdim, ld_g, ld_u = _weights(w_gate, w_up, x.dtype)
    if wdim != dim:
        raise ValueError("x and the weights must have one width")
    shape = (*x.shape[:-1], hidden)
    a, ld_a = _result(out, shape, x.dtype, x, "out")
    gate = up = None
    if isinstance(keep, str):
        if keep == "packed":
            gate, up = _packed8(shape, x), _packed8(shape, x)
        elif keep == "tensors":
            gate, up = x.new_empty(shape), x.new_empty(shape)
        else:
            raise ValueError("keep must be 'tensors', 'packed' or a pair of either")
    elif keep is not None:
        gate, up = keep
    pg, ldg, pu, ldu, g8, u8, held = _kept(gate, up, n, hidden, shape, x)
    dev = _one_device(x, w_gate, w_up, out) if keep is None or isinstance(keep, str) else \
        _one_device(x, w_gate, w_up, out, gate, up)
    if n and hidden:
        if dim == 0:
            raise ValueError("the weights have no columns")
        _call(_abi.lib().zero_gated, dev, _GATED.pack(
            n, dim, hidden, code, kind, x.data_ptr(), ld_x, w_gate.data_ptr(), ld_g, w_up.data_ptr(), ld_u,
            a.data_ptr(), ld_a, pg, ldg, pu, ldu, g8, u8, *_ZEROS[16]))
    return Gated(a, gate, up)


def gated_grad(da: torch.Tensor, gate: Union[torch.Tensor, Packed8], up: Union[torch.Tensor, Packed8], *,
               act: str = "silu", out_gate: Optional[torch.Tensor] = None, out_up: Optional[torch.Tensor] = None,
               again: Union[torch.Tensor, bool] = False) -> GatedGrad:
    """The gradients of gate and up from a's: da * up * act'(gate) and da * act(gate).

    gate, up: what gated kept, as tensors of da's type or in 8 bits.  again: a once more (True,
    or a tensor to write it to), for the gradient of the down projection.  The results
    may lie on da, gate or up.
    """
    n, hidden, ld_da = _rows(da, "da")
    shape, kind, code = da.shape, _act(act), _code(da.dtype)
    pg, ldg, pu, ldu, g8, u8, held = _kept(gate, up, n, hidden, shape, da)
    dg, ld_dg = _result(out_gate, shape, da.dtype, da, "out_gate")
    du, ld_du = _result(out_up, shape, da.dtype, da, "out_up")
    a, ptr_a, ld_a = None, 0, 0
    if again is not False:
        a, ld_a = _result(None if again is True else again, shape, da.dtype, da, "again")
        ptr_a = a.data_ptr()
    dev = _one_device(da, gate, up, out_gate, out_up, again)
    if n and hidden:
        _call(_abi.lib().zero_gated_grad, dev, _GATED.pack(
            n, 0, hidden, code, kind, *_ZEROS[6], ptr_a, ld_a, pg, ldg, pu, ldu, g8, u8, da.data_ptr(), ld_da,
            dg.data_ptr(), ld_dg, du.data_ptr(), ld_du, *_ZEROS[10]))
    return GatedGrad(dg, du, a)


def gated_workspace(tokens: int, dim: int, hidden: int, device="cuda") -> torch.Tensor:
    """A workspace for gated_input_grad and gated_weight_grad calls of at most these
    sizes that do not overlap in time."""
    n = _abi.lib().zero_gated_ws_bytes(tokens, dim, hidden)
    if n == 0:
        raise ValueError("sizes out of range")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _pair(dg: torch.Tensor, du: torch.Tensor):
    if dg.shape != du.shape or dg.dtype != du.dtype:
        raise ValueError("the gradients of gate and up must have one shape and type")
    n, hidden, ld_dg = _rows(dg, "dg")
    return n, hidden, ld_dg, _rows(du, "du")[2]


def gated_input_grad(dg: torch.Tensor, du: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, *,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dx = dg w_gate + du w_up, [..., dim], both products in one kernel."""
    n, hidden, ld_dg, ld_du = _pair(dg, du)
    whid, dim, ld_g, ld_u = _weights(w_gate, w_up, dg.dtype)
    if whid != hidden:
        raise ValueError("the gradients and the weights must have one hidden size")
    code = _code(dg.dtype)
    dx, ld_dx = _result(out, (*dg.shape[:-1], dim), dg.dtype, dg, "out")
    dev = _one_device(dg, du, w_gate, w_up, out, workspace)
    if n == 0 or dim == 0:
        return dx
    if hidden == 0:
        return dx.zero_()
    L = _abi.lib()
    workspace = _workspace(workspace, L.zero_gated_ws_bytes(n, dim, hidden), dg)
    _call(L.zero_gated_input_grad, dev, _GATED.pack(
        n, dim, hidden, code, 0, 0, 0, w_gate.data_ptr(), ld_g, w_up.data_ptr(), ld_u, *_ZEROS[10], dg.data_ptr(), ld_dg,
        du.data_ptr(), ld_du, dx.data_ptr(), ld_dx, *_ZEROS[6], workspace.data_ptr(), workspace.numel()))
    return dx


def gated_weight_grad(dg: torch.Tensor, du: torch.Tensor, x: torch.Tensor, grad_gate: torch.Tensor,
                      grad_up: torch.Tensor, *, accumulate: bool = False,
                      workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """grad_gate = dg^T x and grad_up = du^T x ([hidden, dim], any type), or added to what
    they hold (accumulate).  Returns both."""
    n, hidden, ld_dg, ld_du = _pair(dg, du)
    xn, dim, ld_x = _rows(x, "x")
    if x.shape[:-1] != dg.shape[:-1] or x.dtype != dg.dtype:
        raise ValueError("x and the gradients must have the same rows and type")
    for t, w in ((grad_gate, "grad_gate"), (grad_up, "grad_up")):
        if t.shape != (hidden, dim) or t.dtype != grad_gate.dtype:
            raise ValueError(f"{w} must be [{hidden}, {dim}]; both of one type")
    code, wc = _code(dg.dtype), _code(grad_gate.dtype)
    ld_g, ld_u = _rows(grad_gate, "grad_gate")[2], _rows(grad_up, "grad_up")[2]
    dev = _one_device(dg, du, x, grad_gate, grad_up, workspace)
    if hidden == 0 or dim == 0:
        return grad_gate, grad_up
    L = _abi.lib()
    workspace = _workspace(workspace, L.zero_gated_ws_bytes(n, dim, hidden), dg)
    _call(L.zero_gated_weight_grad, dev, _GATED.pack(
        n, dim, hidden, code, 0, x.data_ptr(), ld_x, *_ZEROS[14], dg.data_ptr(), ld_dg, du.data_ptr(), ld_du, 0, 0,
        grad_gate.data_ptr(), ld_g, grad_up.data_ptr(), ld_u, wc, 1 if accumulate else 0,
        workspace.data_ptr(), workspace.numel()))
    return grad_gate, grad_up

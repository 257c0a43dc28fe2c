"""Plain float64 model of the pre-norm gated feed-forward sub-layer: matrices held in
8 bits, RMS norm, the gated projections, and their backward passes.  Shares no code
with the HIP path.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32


def e4m3(v: np.ndarray) -> np.ndarray:
    """float64 values rounded to the nearest e4m3 number, ties to even (|v| <= 448;
    NaN for NaN and infinities)."""
    v = np.asarray(v, dtype=np.float64)
    out = np.full(v.shape, np.nan)
    ok = np.isfinite(v)
    _, x = np.frexp(np.abs(v[ok]))           # |v| = m 2^x, 1/2 <= m < 1
    step = np.ldexp(1.0, np.maximum(x - 1, -6) - 3)
    out[ok] = np.rint(v[ok] / step) * step   # rint: ties to even
    return out


def e4m3_value(code: np.ndarray) -> np.ndarray:
    """What e4m3 bytes stand for: sign, 4 exponent bits (bias 7), 3 bits of fraction."""
    c = np.asarray(code).astype(np.int64)
    x, f = c >> 3 & 15, c & 7
    mag = np.where(x == 0, f * 2.0 ** -9, (8 + f) * np.exp2(x - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c & 128, -mag, mag)


def blocks(cols: int) -> int:
    return -(-cols // BLOCK)


def hold(v: np.ndarray):
    """[rows, cols] -> (values / scale rounded to e4m3, exponents [rows, blocks])."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    nb = blocks(cols)
    q = np.empty_like(v)
    e = np.empty((rows, nb), dtype=np.int64)
    for b in range(nb):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        top = np.where(np.isfinite(part), np.abs(part), 0.0).max(axis=1)
        m, x = np.frexp(top)
        ex = np.where(m <= 0.875, x - 9, x - 8)          # 448 = 0.875 * 2^9
        e[:, b] = np.maximum(np.where(top == 0, -127, ex), -127)
        q[:, b * BLOCK:(b + 1) * BLOCK] = e4m3(part * np.exp2(-e[:, b].astype(np.float64))[:, None])
    return q, e


def held_value(q: np.ndarray, e: np.ndarray) -> np.ndarray:
    return q * np.exp2(e.astype(np.float64)).repeat(BLOCK, axis=1)[:, :q.shape[1]]


def rms_norm(h, weight, eps):
    """(y, rstd) of [rows, cols]."""
    with np.errstate(divide="ignore", invalid="ignore"):
        rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
        y = h * rstd[:, None]
        return (y if weight is None else y * weight), rstd


def rms_norm_grad(dy, h, rstd, weight, dres=None):
    """(dh, dweight)."""
    n = h * rstd[:, None]
    s = dy if weight is None else dy * weight
    dh = rstd[:, None] * (s - n * (s * n).mean(axis=1, keepdims=True))
    return (dh if dres is None else dh + dres), (dy * n).sum(axis=0)


def act(kind: str, g):
    """act(g), act'(g), and for error bounds p = act(g) / g, the argument z of
    p = 1 / (1 + exp(-z)) and dz / dg."""
    g = np.asarray(g, dtype=np.float64)
    if kind == "silu":
        z, dz = g, np.ones_like(g)
    else:
        k = np.sqrt(2.0 / np.pi)
        z, dz = 2.0 * k * (g + 0.044715 * g ** 3), 2.0 * k * (1.0 + 3.0 * 0.044715 * g * g)
    with np.errstate(over="ignore"):
        p = np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
        one_less = np.where(z >= 0, np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))), 1.0 / (1.0 + np.exp(-np.abs(z))))
    return g * p, p + g * p * one_less * dz, p, z, dz


def gated(x, w_gate, w_up, kind):
    """(a, gate, up)."""
    g, u = x @ w_gate.T, x @ w_up.T
    return act(kind, g)[0] * u, g, u


def gated_grad(da, g, u, kind):
    """(dg, du, a)."""
    v, d = act(kind, g)[:2]
    return da * u * d, da * v, v * u


def products(dg, du, x, w_gate, w_up):
    """(dx, dw_gate, dw_up)."""
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x

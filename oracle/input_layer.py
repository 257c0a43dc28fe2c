"""Plain float64 model of the input layer: embedding lookup, its gradient, and
counter-based dropout.  Shares no code with the HIP path.

Philox4x32-10 is written from the published algorithm (Salmon, Moraes, Dror and
Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11).
"""
from __future__ import annotations

import numpy as np

U32 = np.uint64(0xFFFFFFFF)


def philox4x32(ctr, key, rounds: int = 10):
    """ctr: four uint32 arrays, key: two uint32 numbers -> four uint64 arrays < 2^32."""
    c = [np.asarray(x).astype(np.uint64) & U32 for x in ctr]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(rounds):
        p0 = c[0] * np.uint64(0xD2511F53)
        p1 = c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & U32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & U32]
        k0 = (k0 + 0x9E3779B9) & 0xFFFFFFFF
        k1 = (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def threshold(p: float) -> int:
    return int(np.rint(np.float64(p) * 65536.0))


def keep_scale(p: float) -> float:
    t = threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def keep(rows: int, cols: int, p: float, seed: int, site: int, step: int, row0: int = 0) -> np.ndarray:
    """[rows, cols] truth values: element kept."""
    g = (cols + 7) // 8
    c0 = np.broadcast_to(np.arange(g, dtype=np.uint64), (rows, g))
    c1 = np.broadcast_to((np.arange(rows, dtype=np.uint64) + np.uint64(row0))[:, None], (rows, g))
    c2 = np.full((rows, g), step & 0xFFFFFFFF, dtype=np.uint64)
    c3 = np.full((rows, g), site, dtype=np.uint64)
    w = philox4x32((c0, c1, c2, c3), (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    u = np.empty((rows, g, 8), dtype=np.int64)
    for j in range(4):
        u[:, :, 2 * j] = (w[j] & np.uint64(0xFFFF)).astype(np.int64)
        u[:, :, 2 * j + 1] = (w[j] >> np.uint64(16)).astype(np.int64)
    return u.reshape(rows, g * 8)[:, :cols] >= threshold(p)


def _drop(y: np.ndarray, drop) -> np.ndarray:
    if drop is None:
        return y
    k = keep(y.shape[0], y.shape[1], **drop)
    return np.where(k, y * keep_scale(drop["p"]), 0.0)


def dropout(x: np.ndarray, drop, residual=None) -> np.ndarray:
    y = _drop(np.asarray(x, dtype=np.float64), drop)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)


def lookup(ids, table, scale=1.0, id0=0, pos_table=None, pos=None, pos_period=0, drop=None) -> np.ndarray:
    """ids: sequence of integers; table [rows, dim]."""
    rows, dim = table.shape
    y = np.zeros((len(ids), dim))
    for t, i in enumerate(int(i) for i in ids):
        if id0 <= i < id0 + rows:
            y[t] = np.float64(scale) * np.asarray(table[i - id0], dtype=np.float64)
        if pos_table is not None:
            q = int(pos[t]) if pos is not None else t % pos_period
            if 0 <= q < pos_table.shape[0]:
                y[t] += np.asarray(pos_table[q], dtype=np.float64)
    return _drop(y, drop)


def lookup_grad(dy, ids, rows, scale=1.0, id0=0, period=0, drop=None):
    """Gradient [rows, dim], and per row the number of terms and their absolute sum
    (what the error bound of an fp32 sum needs)."""
    g = _drop(np.asarray(dy, dtype=np.float64), drop) * np.float64(scale)
    out = np.zeros((rows, g.shape[1]))
    mag = np.zeros_like(out)
    cnt = np.zeros(rows, dtype=np.int64)
    for t in range(g.shape[0]):
        v = (t % period if ids is None else int(ids[t])) - id0
        if 0 <= v < rows:
            out[v] += g[t]
            mag[v] += np.abs(g[t])
            cnt[v] += 1
    return out, cnt, mag

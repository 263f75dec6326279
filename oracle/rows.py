"""Norm and rotation of query / key heads, and rows in and out of the paged cache, in float64 from
their definitions (test infrastructure only).

Rows x [tokens, heads, d]; table [max_pos, rot]: cosines, then sines.  A negative position is
padding: its rows come back as NaN (not written) from the forward, as 0 from the backward."""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode

E4M3_MAX = 448.0


def e4m3_round(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even, saturating at +-448; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(x)))
        step = np.exp2(np.maximum(np.where(np.isfinite(e), e, -6.0), -6.0) - 3.0)
        y = np.clip(np.rint(x / step) * step, -E4M3_MAX, E4M3_MAX)
    return np.where(np.isinf(x), np.sign(x) * E4M3_MAX, y)


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, table, positions, interleaved=False, back=False):
    y = np.array(x, dtype=np.float64)
    if table is None:
        return y
    rot = table.shape[1]
    ia, ib = _pairs(rot, interleaved)
    row = np.asarray(table, dtype=np.float64)[np.maximum(positions, 0)][:, None, :]
    c, s = row[..., : rot // 2], row[..., rot // 2 :] * (-1.0 if back else 1.0)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def norm_rope(x, weight, table, positions, eps, norm=True, interleaved=False):
    x = np.asarray(x, dtype=np.float64)
    y = x
    if norm:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * np.asarray(weight, dtype=np.float64)
    y = rotate(y, table, positions, interleaved)
    if positions is not None:
        y[np.asarray(positions) < 0] = np.nan
    return y


def norm_rope_backward(dy, x, weight, table, positions, eps, norm=True, interleaved=False):
    """(dx, dweight); dweight is None without the norm."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    g = rotate(dy, table, positions, interleaved, back=True)
    if positions is not None:
        g[np.asarray(positions) < 0] = 0.0
    if not norm:
        return g, None
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = np.where(g == 0.0, 0.0, x * r) if positions is not None else x * r
    u = g * w
    dx = r * (u - x * r * (u * n).mean(-1, keepdims=True))
    if positions is not None:
        dx[np.asarray(positions) < 0] = 0.0
    return dx, (g * n).sum((0, 1))


def row_places(cu, seq_lens, block_table, block_size):
    """(row, request, position, block, slot) of every packed row."""
    out = []
    for r in range(len(seq_lens)):
        n = int(cu[r + 1]) - int(cu[r])
        for j in range(n):
            p = int(seq_lens[r]) - n + j
            out.append((int(cu[r]) + j, r, p, int(block_table[r][p // block_size]), p % block_size))
    return out


def quantise_row(x):
    """(scale, values of the codes) of one row of fp32-representable values: the scale and the
    quotients are rounded to fp32, as the format's definition has them."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.float32(np.nan) if np.isnan(x).any() else np.abs(x).max()
        scale = np.float32(amax / np.float32(E4M3_MAX))
        q = x / scale if scale > 0 else np.zeros_like(x)
    return scale, e4m3_round(q)


def cache_gates(log_gate, g_cache, cu, seq_lens, block_table, block_size):
    """g_cache (float64 copy) after the append of log_gate [rows, hq]."""
    g = np.array(g_cache, dtype=np.float64)
    for t, r, p, blk, slot in row_places(cu, seq_lens, block_table, block_size):
        prev = 0.0
        if p > 0:
            prev = g[int(block_table[r][(p - 1) // block_size]), :, (p - 1) % block_size]
        g[blk, :, slot] = prev + np.asarray(log_gate, dtype=np.float64)[t]
    return g


def cache_gather(cache, scale, cu, seq_lens, block_table, block_size):
    """Rows [rows, hkv, d] of one cache [blocks, hkv, slots, d]: codes (uint8, with per-token or
    one-element scale) or values (scale None); products in float64."""
    n = int(cu[len(seq_lens)])
    out = np.zeros((n, cache.shape[1], cache.shape[3]))
    for t, _, _, blk, slot in row_places(cu, seq_lens, block_table, block_size):
        if scale is None:
            out[t] = cache[blk, :, slot]
        else:
            sc = np.asarray(scale, dtype=np.float64)
            sc = sc.reshape(1, 1) if sc.size == 1 and sc.ndim == 1 else sc[blk, :, slot][:, None]
            out[t] = e4m3_decode(cache[blk, :, slot]) * sc
    return out

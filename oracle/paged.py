"""A paged K/V cache, restated in float64 NumPy: the rotation of positions, where a
position lies, and attention over the pages."""

from __future__ import annotations

import numpy as np


def rope_table(n_pos: int, rot: int, base: float = 10000.0) -> np.ndarray:
    """[n_pos][rot] float32: rot / 2 cosines, then rot / 2 sines."""
    a = np.arange(n_pos)[:, None] * base ** (-np.arange(rot // 2) / max(1, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate(x, rope_rows, rot: int, neighbours: bool) -> np.ndarray:
    """x [n, heads, d], rope_rows [n, rot] -> float64 [n, heads, d]."""
    y = np.array(x, np.float64)
    c, s = np.asarray(rope_rows, np.float64)[:, None, :rot // 2], np.asarray(rope_rows, np.float64)[:, None, rot // 2:]
    ia = np.arange(0, rot, 2) if neighbours else np.arange(rot // 2)
    ib = ia + (1 if neighbours else rot // 2)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def slots(pages, page: int, first: int, count: int) -> np.ndarray:
    """Slots of positions first .. first + count - 1 of a request with these pages."""
    t = np.arange(first, first + count)
    return np.asarray(pages, np.int64)[t // page] * page + t % page


def attention(q, k, v, ctx: int, scale: float):
    """q [n, heads, d], k, v [kv_heads, keys, d]: row j sees keys 0 .. ctx + j.  Returns out [n, heads, d] and
    spread [n, heads, d] = sqrt(sum_t w_t^2 (v_t - out)^2), by which independent relative errors of the weights move it."""
    n, heads, d = q.shape
    group = heads // k.shape[0]
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(heads):
        kk, vv = k[h // group].astype(np.float64), v[h // group].astype(np.float64)
        s = q[:, h].astype(np.float64) @ kk.T * scale
        s = np.where(np.arange(kk.shape[0])[None] <= ctx + np.arange(n)[:, None], s, -np.inf)
        w = np.exp(s - s.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        out[:, h] = w @ vv
        w2 = w * w
        spread[:, h] = np.sqrt(np.maximum(w2 @ (vv * vv) - 2 * out[:, h] * (w2 @ vv) + out[:, h] ** 2 *
                                          w2.sum(1, keepdims=True), 0))
    return out, spread

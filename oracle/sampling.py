"""Sampling one token from a row of logits with a given uniform number, in float64 NumPy."""

from __future__ import annotations

import numpy as np


def sample(row, u: float, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0) -> int:
    """-1 where nothing can be drawn.  Arguments are taken at the float32 values the GPU sees."""
    u, temperature, top_p, min_p = (float(np.float32(x)) for x in (u, temperature, top_p, min_p))
    x = np.asarray(row, np.float32).astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1
    if temperature == 0:
        return int(np.argmax(x))
    with np.errstate(all="ignore"):
        w = np.where(x == top, 1.0, np.exp((x - top) / temperature))
    order = np.lexsort((np.arange(len(x)), -x))  # descending, ids ascending on ties
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1:
        mass = np.cumsum(w[order])
        order = order[:max(1, int(np.searchsorted(mass, top_p * mass[-1], side="left")) + 1)]
    order = np.sort(order[w[order] >= min_p])
    mass = np.cumsum(w[order])
    return int(order[int(np.searchsorted(mass, u * mass[-1], side="right"))])

"""A K/V cache held in 4 bits, restated in float64 NumPy: the codes of a row, the
bytes of a layer, the values they stand for, and attention over them."""

from __future__ import annotations

import numpy as np


def bf16(a) -> np.ndarray:
    """float32 to the nearest bf16 (ties to even), as float32; overflow goes to infinity, NaN stays."""
    a = np.ascontiguousarray(a, np.float32)
    u = a.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(a), a, r).astype(np.float32)


def quantise(x):
    """x [..., d] float32 -> codes [..., d] uint8, scale and minimum [..., G] float32 (bf16 values)."""
    x = np.ascontiguousarray(x, np.float32)
    d = x.shape[-1]
    G = max(1, d // 32)
    g = x.reshape(x.shape[:-1] + (G, d // G))
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # (NaN if any is)
        s, m = bf16((hi - lo) / np.float32(15)), bf16(lo)
        bad = ~(np.isfinite(s) & np.isfinite(m))
        s, m = np.where(bad, np.float32(np.nan), s), np.where(bad, np.float32(np.nan), m)
        q = (g.astype(np.float64) - m[..., None]) / s[..., None]
        c = np.where((s > 0)[..., None], np.clip(np.rint(q), 0, 15), 0).astype(np.uint8)
    return c.reshape(x.shape), s.astype(np.float32), m.astype(np.float32)


def stands_for(c, s, m) -> np.ndarray:
    d, G = c.shape[-1], s.shape[-1]
    return (np.repeat(m, d // G, -1).astype(np.float64) + np.repeat(s, d // G, -1).astype(np.float64) * c)


def _param(s, m):
    u = np.ascontiguousarray(s).view(np.uint32) >> 16 | (np.ascontiguousarray(m).view(np.uint32) & 0xFFFF0000)
    return u.astype(np.uint32)


class Layer:
    """The bytes of one layer."""

    def __init__(self, n_heads, d, kv_slots, data: np.ndarray):
        self.S, self.G = (kv_slots + 15) // 16 * 16, max(1, d // 32)
        self.d = d
        S, G = self.S, self.G
        codes, params = n_heads * S * d // 2, n_heads * S * G * 4
        assert data.size == 2 * (codes + params)
        self.kc = data[:codes].reshape(n_heads, S, d // 2)
        self.vc = data[codes:2 * codes].view(np.uint16).reshape(n_heads, S // 2, d // 4, 2)
        self.kp = data[2 * codes:2 * codes + params].view(np.uint32).reshape(n_heads, S, G)
        self.vp = data[2 * codes + params:].view(np.uint32).reshape(n_heads, S // 2, G, 2)

    def write(self, slot: int, k, v):
        """k, v [n_heads, d] of one slot."""
        c, s, m = quantise(k)
        self.kc[:, slot] = c[:, 0::2] | c[:, 1::2] << 4
        self.kp[:, slot] = _param(s, m)
        c, s, m = quantise(v)
        c = c.astype(np.uint16)
        self.vc[:, slot // 2, :, slot % 2] = c[:, 0::4] | c[:, 1::4] << 4 | c[:, 2::4] << 8 | c[:, 3::4] << 12
        self.vp[:, slot // 2, :, slot % 2] = _param(s, m)

    @staticmethod
    def _split(p):
        return (p << 16).astype(np.uint32).view(np.float32), (p & np.uint32(0xFFFF0000)).view(np.float32)

    def read(self, first: int, count: int):
        """k, v [n_heads, count, d] float64."""
        kc = np.stack([self.kc[:, first:first + count] & 15, self.kc[:, first:first + count] >> 4], -1)
        k = stands_for(kc.reshape(kc.shape[:2] + (self.d,)), *self._split(self.kp[:, first:first + count]))
        at = np.arange(first, first + count)
        w = self.vc[:, at // 2, :, at % 2].transpose(1, 0, 2)
        vc = np.stack([w >> (4 * i) & 15 for i in range(4)], -1).reshape(w.shape[:2] + (self.d,))
        v = stands_for(vc, *self._split(np.ascontiguousarray(self.vp[:, at // 2, :, at % 2].transpose(1, 0, 2))))
        return k, v


def attention(q, k, v, ctx: int) -> np.ndarray:
    """q [n, heads, d], k, v [heads, keys, d] -> [n, heads, d]: row j sees keys 0 .. ctx + j."""
    d = q.shape[-1]
    out = np.zeros(q.shape)
    for j in range(q.shape[0]):
        s = np.einsum("hd,hkd->hk", q[j].astype(np.float64), k[:, :ctx + j + 1]) / np.sqrt(d)
        p = np.exp(s - s.max(-1, keepdims=True))
        out[j] = np.einsum("hk,hkd->hd", p / p.sum(-1, keepdims=True), v[:, :ctx + j + 1])
    return out

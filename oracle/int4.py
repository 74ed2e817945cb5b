"""4-bit cache rows for the oracle (test infrastructure).

A row holds the D elements of one token and KV head in D / 32 groups of 32: per group a step
and a minimum in fp16, per element a code n in 0..15, value = minimum + step * n (times the
tensor's scale). Bytes: D/2 of codes (32-bit little-endian words of eight; the word of
elements 32 g + 8 t .. + 7 is word t * (D/32) + g, element j of the eight in bits 4 j), then
the steps, then the minima. Writing a row rounds the minimum down and the step, a fifteenth
of the range above the minimum, up, and takes the nearest code (ties to even). Values saturate
at +-65280, so that every value a row holds rounds to a finite fp16. A group that
holds a NaN or an infinity has NaN (0x7fff) for both.
"""
from __future__ import annotations

import numpy as np


def row_bytes(D: int) -> int:
    return D // 2 + 4 * (D // 32)


def unpack(rows: np.ndarray):
    """(codes [..., G, 32] int, steps [..., G] float64, minima [..., G] float64) of uint8 rows."""
    D = rows.shape[-1] * 8 // 5
    G = D // 32
    rows = np.ascontiguousarray(rows)
    words = rows[..., :D // 2].copy().view("<u4").reshape(*rows.shape[:-1], 4, G)
    codes = np.zeros(rows.shape[:-1] + (G, 32), dtype=np.int64)
    for t in range(4):
        for j in range(8):
            codes[..., 8 * t + j] = (words[..., t, :] >> np.uint32(4 * j)) & np.uint32(15)
    meta = rows[..., D // 2:].copy().view("<f2").astype(np.float64)
    return codes, meta[..., :G], meta[..., G:]


def pack(codes: np.ndarray, steps: np.ndarray, minima: np.ndarray) -> np.ndarray:
    """uint8 rows of codes [..., G, 32] and fp16 steps and minima [..., G]."""
    G = codes.shape[-2]
    words = np.zeros(codes.shape[:-2] + (4, G), dtype="<u4")
    for t in range(4):
        for j in range(8):
            words[..., t, :] |= codes[..., 8 * t + j].astype("<u4") << np.uint32(4 * j)
    lead = codes.shape[:-2]
    words = np.ascontiguousarray(words).reshape(*lead, 4 * G).view(np.uint8)
    meta = np.concatenate([steps, minima], axis=-1).astype("<f2")
    return np.concatenate([words, np.ascontiguousarray(meta).view(np.uint8)], axis=-1)


def dequant(rows: np.ndarray, scale: float = 1.0) -> np.ndarray:
    """Values [..., D] in float64 of uint8 rows."""
    codes, steps, minima = unpack(rows)
    x = minima[..., None] + steps[..., None] * codes
    return x.reshape(*rows.shape[:-1], -1) * float(np.float32(scale))


def _half(x: np.ndarray, up: bool) -> np.ndarray:
    """x rounded up (down) to fp16; |x| <= 65280."""
    h = x.astype(np.float16)
    w = h.astype(np.float64)
    return np.where((w < x) if up else (w > x),
                    np.nextafter(h, np.float16(65504.0 if up else -65504.0)), h)


def quantise(x: np.ndarray) -> np.ndarray:
    """uint8 rows that hold x [..., D] (float64, already divided by the scale)."""
    g = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(g).all(-1)           # such a group reads back as NaN
    g = np.clip(np.where(bad[..., None], 0.0, g), -65280.0, 65280.0)
    minima = _half(g.min(-1), up=False)
    low = minima.astype(np.float64)
    steps = _half((g.max(-1) - low) / 15.0, up=True)
    st = steps.astype(np.float64)[..., None]
    n = np.where(st > 0, (g - low[..., None]) / np.where(st > 0, st, 1.0), 0.0)
    nan = np.array(0x7FFF, dtype=np.uint16).view(np.float16)
    return pack(np.clip(np.rint(n), 0, 15).astype(np.int64), np.where(bad, nan, steps),
                np.where(bad, nan, minima))

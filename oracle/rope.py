"""Rotary positions for the oracle (test infrastructure): the definition in float64."""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim: int, base: float = 10000.0, kind=None, factor: float = 1.0,
                original_max: int = 0, slow: float = 1.0, fast: float = 32.0):
    """(radians per token of each pair [rot_dim / 2], amplitude)."""
    n = rot_dim // 2
    if kind == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = np.array([base ** (-i / n) for i in range(n)])
    if kind in (None, "ntk"):
        return f, 1.0
    if kind == "linear":
        return f / factor, 1.0
    turns = original_max * f / (2 * math.pi)       # over the original context
    if kind == "banded":
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    assert kind == "yarn"
    # the (real) pair index that makes a given number of turns
    at = lambda t: n * math.log(original_max / (2 * math.pi * t)) / math.log(base)
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot_dim - 1)
    ramp = np.clip((np.arange(n) - lo) / max(hi - lo, 1e-3), 0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1


def rotate(x: np.ndarray, pos: np.ndarray, freq: np.ndarray, interleaved: bool = False,
           amplitude: float = 1.0) -> np.ndarray:
    """x [T, H, D] with the first 2 len(freq) elements of each head turned to positions pos [T]."""
    x = np.asarray(x, dtype=np.float64)
    n = len(freq)
    z = x[..., 0:2 * n:2] + 1j * x[..., 1:2 * n:2] if interleaved else x[..., :n] + 1j * x[..., n:2 * n]
    z = z * (amplitude * np.exp(1j * (np.asarray(pos, np.float64)[:, None] * freq)))[:, None, :]
    y = x.copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y

"""Shared by the tests of cross attention and of decode behind shared prefixes: seeded paged
caches whose unwritten slots hold NaN, the definitions in 64 bits, and bounds on the error.

Bounds. An output is sum_t w_t v_t with weights w_t >= 0 that sum to 1. Relative to w_t, the kernel's
weight is off by
  u_p                      its rounding to the type of the products (half a step), and
  e = ln 2 * (error of the exponent, in log2 units) + 2^-21
with the exponent's error from D fp32 sums of a dot product of size S_t = sum_d |q_d k_d| (each at
most 2^-24 of the running sum, which S_t bounds), the scale's rounding and the product's, at most
(D + 3) 2^-24 |scale| log2(e) max_t S_t, and the approximation of 2^x and the rescalings at most
2^-21. Weights enter the sums of up to L terms in fp32, off by at most 2^-24 of the sum of magnitudes
per term, and the denominator likewise: (2 L) 2^-24 is a bound that no order of the sums exceeds.
So |out - exact| <= u_o |exact| + (u_p + 2 e + 2 L 2^-24) sum_t w_t |v_t| + fp16's smallest step for
weights that are subnormal there (2^-25 each, where the largest weight of the row is at least 2^-2)
and for the output.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import e4m3_to_float64

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8 / 1, "f16": 2.0 ** -11}
SCALE8 = 5.0 / 448.0


class Pool:
    """Paged caches of B sequences. prefixes: [(first, end, tokens)] groups whose sequences share
    leading tokens: whole blocks through the first's table, a block that the prefix ends in copied
    (own_prefix=True), or the members' tables holding -1 and their own copies NaN (False: only the
    first sequence's are ever read)."""

    def __init__(self, lens, Hkv, D, bs, dtype="bf16", cache="same", seed=0, prefixes=(), own_prefix=True,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.bs, self.cache, self.dtype = list(lens), Hkv, D, bs, cache, dtype
        B = len(lens)
        need = [-(-L // bs) for L in lens]
        pool = sum(need) + 3
        perm = torch.randperm(pool, generator=g).tolist()
        self.bt = torch.full((B, max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.bt[b, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        K = [spread * torch.randn(L, Hkv, D, generator=g) for L in lens]
        V = [torch.randn(L, Hkv, D, generator=g) for L in lens]
        for a, e, P in prefixes:
            for b in range(a + 1, e):
                n = min(P, lens[a], lens[b])
                K[b][:n], V[b][:n] = K[a][:n], V[a][:n]
        self.scale = SCALE8 if cache == "fp8" else 1.0
        store = (lambda x: (x / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn)) if cache == "fp8" else \
            (lambda x: x.to(DT[dtype]))
        wide = (lambda x: e4m3_to_float64(x.view(torch.uint8).numpy()) * float(np.float32(SCALE8))) \
            if cache == "fp8" else (lambda x: x.double().numpy())
        self.K, self.V, self.caches = [], [], []
        for X, out in ((K, self.K), (V, self.V)):
            c = store(torch.full((pool, bs, Hkv, D), float("nan")))
            raw = c.view(torch.uint8 if cache == "fp8" else torch.int16)
            for b, L in enumerate(lens):
                rows = store(X[b])
                out.append(wide(rows))
                pos = torch.arange(L)
                keep = torch.ones(L, dtype=torch.bool)
                if not own_prefix:
                    for a, e, P in prefixes:
                        if a < b < e:
                            keep[:min(P, lens[a], L)] = False
                pos = pos[keep]
                raw[self.bt[b, pos // bs].long(), pos % bs] = rows.view(raw.dtype)[keep]
            self.caches.append(c)
        if own_prefix:
            for a, e, P in prefixes:  # whole blocks of the prefix through the first's table
                n = min(P, lens[a]) // bs
                for b in range(a + 1, e):
                    self.bt[b, :min(n, need[b])] = self.bt[a, :min(n, need[b])]
        else:
            for a, e, P in prefixes:
                for b in range(a + 1, e):
                    self.bt[b, :min(min(P, lens[a]), lens[b]) // bs] = -7

    def cuda(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        return (self.caches[0].cuda(), self.caches[1].cuda(), self.bt.cuda(), i32(self.lens))


def queries(shape, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed + 77)
    return (spread * torch.randn(shape, generator=g)).to(DT[dtype])


def attend(q, K, V, scale, lim=None):
    """q [n, Hq, D], K, V [L, Hkv, D] in float64; row i sees t < lim[i] (all without lim). Returns
    (out, sum_t w |v|, max_t S_t), the last for the bound."""
    n, Hq, D = q.shape
    L, Hkv = K.shape[0], K.shape[1]
    G = Hq // Hkv
    out, mag, size = np.zeros_like(q), np.zeros_like(q), 0.0
    if L == 0 or n == 0:
        return out, mag, size
    for h in range(Hq):
        k, v = K[:, h // G], V[:, h // G]
        s = float(scale) * (q[:, h] @ k.T)
        if lim is not None:
            s = np.where(np.arange(L)[None, :] < np.asarray(lim)[:, None], s, -np.inf)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
        den = e.sum(-1, keepdims=True)
        w = e / np.where(den > 0, den, 1.0)
        out[:, h], mag[:, h] = w @ v, w @ np.abs(v)
        size = max(size, float((np.abs(q[:, h]) @ np.abs(k).T).max()))
    return out, mag, size


def check(got, ref, mag, size, pool, scale, what=""):
    y = got.detach().double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(y).all(), f"{what}: not finite"
    L = max(pool.lens + [1])
    prod = "f16" if pool.cache == "fp8" else pool.dtype
    e = math.log(2) * (pool.D + 3) * 2.0 ** -24 * abs(scale) * math.log2(math.e) * size + 2.0 ** -21
    tiny = 2.0 ** -24 + (2.0 ** -23 * L * max(1.0, np.abs(pool.V[0]).max() if len(pool.V[0]) else 1.0) * 2.0 ** -8
                         if prod == "f16" else 0.0)
    tol = HALF_STEP[pool.dtype] * np.abs(ref) + (HALF_STEP[prod] + 2 * e + 2 * L * 2.0 ** -24) * mag + tiny
    bad = np.abs(y - ref) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} beyond the bound, worst {np.max(np.abs(y - ref) / tol):.3g} times it, at {np.argwhere(bad)[:3].tolist()}"

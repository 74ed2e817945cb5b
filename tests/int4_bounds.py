"""Decode over 4-bit caches: inputs whose every token can be made to count, the float64
reference, and bounds that follow from each element's own terms."""
from __future__ import annotations

import math

import numpy as np
import torch

import rows_harness as rh
from oracle import int4 as o4

# Significant bits of the output types.
BITS = {"bf16": 8, "f16": 11}


def spread(x, dtype):
    """Quadratic mean of the error with which values near x round to dtype: a step / sqrt(12)."""
    _, e = np.frexp(x)
    return 2.0 ** (np.maximum(e, -13) - BITS[dtype]) / math.sqrt(12)


class Case:
    """One call's inputs. heavy: tokens (of each sequence that has them; negative ones count
    from its end) that the queries prefer to all others together."""

    def __init__(self, lens, Hq, Hkv, D, bs, dtype="bf16", rows=1, window=0, seed=0, heavy=(), k_scale=1.0,
                 v_scale=1.0):
        self.lens, self.Hq, self.Hkv, self.D, self.bs = list(lens), Hq, Hkv, D, bs
        self.dtype, self.rows, self.window = dtype, rows, window
        self.k_scale, self.v_scale = float(np.float32(k_scale)), float(np.float32(v_scale))
        self.scale = float(np.float32(1 / math.sqrt(D) / self.k_scale))
        self.kc, self.vc, self.bt, _, _ = rh.random_int4_pool(lens, bs, Hkv, D, seed, spread=0.3)
        g = np.random.default_rng(seed + 99)
        B, G = len(lens), Hq // Hkv
        u = g.standard_normal((B, 1, Hkv, 1, D))
        q = u + 0.2 * g.standard_normal((B, rows, Hkv, G, D))
        self.q = torch.from_numpy(q.reshape((B, Hq, D) if rows == 1 else (B, rows, Hq, D)).astype(np.float32)).to(
            rh.DT[dtype])
        for b, L in enumerate(lens):
            pos = sorted({t if t >= 0 else L + t for t in heavy if -L <= t < L})
            if pos:
                p = torch.tensor(pos)
                c = (math.log(L) + 1.5) / math.sqrt(D)
                rows4 = torch.from_numpy(o4.quantise(np.repeat(c * u[b, 0, None, :, 0], len(pos), 0)))
                self.kc[self.bt[b, p // bs].long(), :, p % bs] = rows4

    def rows_of(self, cache, b):
        return rh.cache_rows(cache, "int4", self.bt, b, np.arange(self.lens[b]), self.bs).numpy()

    def reference(self, drop=None, zero_v=None):
        """(outputs, element bounds), both [B, R, Hq, D] in float64. drop, zero_v (for tests of
        the bounds): b, L -> tokens of sequence b that are left out, whose values are zero."""
        B, R, G, D = len(self.lens), self.rows, self.Hq // self.Hkv, self.D
        q = rh.f64(self.q).reshape(B, R, self.Hkv, G, D)
        ref, tol, var = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
        half = rh.HALF_STEP[self.dtype]
        for b, L in enumerate(self.lens):
            if L == 0:
                continue
            kr, vr = self.rows_of(self.kc, b), self.rows_of(self.vc, b)
            K, V = o4.dequant(kr) * self.k_scale, o4.dequant(vr) * self.v_scale
            n, st, _ = o4.unpack(vr)
            most = (st[..., None] * np.maximum(n, 15 - n)).reshape(V.shape) * self.v_scale
            mean2 = (st[..., None] ** 2 * (n ** 2 + (15 - n) ** 2) / 2).reshape(V.shape) * self.v_scale ** 2
            _, kst, kmn = o4.unpack(kr)
            ksize = np.repeat((np.abs(kmn) + 15 * kst) * self.k_scale, 32, axis=-1)
            gone = np.zeros(L, bool)
            if drop is not None:
                gone[drop(b, L)] = True
            if zero_v is not None:
                V = V.copy()
                V[zero_v(b, L)] = 0
            for i in range(R):
                hi = L - R + i + 1
                lo = max(0, L - self.window) if self.window else 0
                if hi <= lo:
                    continue
                see = np.arange(lo, hi)[~gone[lo:hi]]
                if not len(see):
                    continue
                for h in range(self.Hkv):
                    qh, v = q[b, i, h], V[see, h]
                    s = self.scale * qh @ K[see, h].T
                    e = np.exp(s - s.max(1, keepdims=True))
                    den = e.sum(1, keepdims=True)
                    w = e / den
                    out = w @ v
                    # a score's fp32 sums: 16 roundings and cuts of 2^-23 of at most its terms' sizes; the
                    # exponential 2^-21
                    off = 2.0 ** -19 * self.scale * np.abs(qh) @ ksize[see, h].T + 2.0 ** -21
                    ref[b, i, h] = out
                    tol[b, i, h] = (half * np.abs(out)
                                    + 2.0 ** -11 * (w @ (np.abs(v) + most[see, h]))      # weights, products
                                    + 2.0 ** -25 * (np.abs(v) + 15 * self.v_scale).sum(0) / den  # ... below fp16's normal range
                                    + (w * off) @ np.abs(v) + (w * off).sum(1, keepdims=True) * np.abs(out)
                                    # sums of a warp's tokens (a quarter of all at most), 3 cuts of 2^-23 per 16
                                    + 3 * (hi - lo + 128) / 64 * 2.0 ** -23 * 2 * (w @ most[see, h]))
                    # for the norm: the output's rounding; a weight's, one for all elements, taken
                    # at its worst; a product's, one for a group, spread over its half step
                    var[b, i, h] = spread(out, self.dtype) ** 2 + 2.0 ** -22 * (
                        w ** 2 @ v ** 2 + w ** 2 @ mean2[see, h] / 3)
        shape = (B, R, self.Hq, D)
        if drop is None and zero_v is None:
            self.norm_tol = 1.3 * np.sqrt(var.reshape(shape).sum((2, 3)))   # room for how a draw falls
        return ref.reshape(shape), tol.reshape(shape)

    def errors(self, got, ref, tol):
        """(worst element error over its bound, worst norm error of a sequence's row over its bound)."""
        got = np.asarray(got, np.float64).reshape(ref.shape)
        worst = float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()) if got.size else 0.0
        norm = np.sqrt(((got - ref) ** 2).sum((2, 3))) / np.maximum(self.norm_tol, 1e-300)
        return worst, float(norm.max())

    def decode(self, pa, workspace, **kw):
        return pa.decode(self.q.cuda(), self.kc.cuda(), self.vc.cuda(), self.bt.cuda(),
                         torch.tensor(self.lens, dtype=torch.int32, device="cuda"), self.scale,
                         max_seq_len=max(self.lens + [1]), window=self.window, k_scale=self.k_scale,
                         v_scale=self.v_scale, workspace=workspace, **kw)

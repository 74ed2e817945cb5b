"""Shared by the tests of append, gather and decode over 4-bit caches: seeded pools, tables
and lengths, and the oracle's view of them."""
from __future__ import annotations

import numpy as np
import torch

from oracle import e4m3_to_float64
from oracle import int4 as o4
from oracle import rope as orope

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
# half a step of each type, relative to the value
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def tables_for(lens, bs, seed, spare=3):
    """(block_tables with -1 past each sequence, blocks in the pool)."""
    rng = np.random.default_rng(seed)
    need = [-(-L // bs) for L in lens]
    pool = sum(need) + spare
    perm = rng.permutation(pool)
    bt = np.full((len(lens), max(need + [1])), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(bt), pool


def empty_pool(cache, pool, bs, Hkv, D, dtype, seed, nan=True):
    """A cache pool whose every slot holds NaN (or noise): unwritten slots must not matter."""
    rng = np.random.default_rng(seed)
    if cache == "int4":
        rows = rng.integers(0, 256, (pool, Hkv, bs, o4.row_bytes(D)), dtype=np.uint8)
        if nan:
            rows[..., D // 2:] = np.frombuffer(np.float16(np.nan).tobytes(), np.uint8)[None].repeat(
                rows[..., D // 2:].shape[-1] // 2, 0).reshape(-1)
        return torch.from_numpy(rows)
    x = torch.full((pool, bs, Hkv, D), float("nan") if nan else 0.5)
    return x.to(torch.float8_e4m3fn if cache == "fp8" else DT[dtype])


def bits(t: torch.Tensor) -> torch.Tensor:
    """The tensor's raw bytes, comparable with torch.equal (NaN included)."""
    return t.detach().cpu().contiguous().view(torch.uint8)


def cache_rows(cache_tensor, kind, bt, b, pos, bs):
    """Raw rows [len(pos), Hkv, row] of sequence b's tokens, on the CPU."""
    c = cache_tensor.detach().cpu()
    phys = bt[b, torch.as_tensor(pos) // bs].long()
    slot = torch.as_tensor(pos) % bs
    if kind == "int4":
        return c[phys, :, slot]
    if kind == "fp8":
        return c.view(torch.uint8)[phys, slot]
    return c[phys, slot]


def values(rows: torch.Tensor, kind: str, scale: float = 1.0) -> np.ndarray:
    """float64 values of raw rows."""
    if kind == "int4":
        return o4.dequant(rows.numpy(), scale)
    if kind == "fp8":
        return e4m3_to_float64(rows.numpy()) * float(np.float32(scale))
    return f64(rows)


def positions(lens, starts, R, B):
    """[(row, sequence, position)] of the rows of a call that belong to a sequence."""
    out = []
    for b in range(B):
        r0, n = (starts[b], starts[b + 1] - starts[b]) if starts is not None else (b * R, R)
        out += [(r0 + i, b, lens[b] - n + i) for i in range(n)]
    return out


def random_int4_pool(lens, bs, Hkv, D, seed, step=0.3, spread=1.0):
    """A 4-bit pool with known contents: (k_cache, v_cache, tables, K, V), K[b] [L, Hkv, D] in
    float64. Slots that hold no token are NaN."""
    rng = np.random.default_rng(seed)
    bt, pool = tables_for(lens, bs, seed + 1)
    caches, vals = [], []
    G = D // 32
    for which in range(2):
        c = empty_pool("int4", pool, bs, Hkv, D, "bf16", seed + 2 + which)
        per = []
        for b, L in enumerate(lens):
            codes = rng.integers(0, 16, (L, Hkv, G, 32))
            st = (step * np.exp(spread * 0.5 * rng.standard_normal((L, Hkv, G)))).astype(np.float16)
            mn = (-7.5 * st.astype(np.float64) + 0.2 * rng.standard_normal(st.shape)).astype(np.float16)
            rows = o4.pack(codes, st, mn)
            pos = torch.arange(L)
            c[bt[b, pos // bs].long(), :, pos % bs] = torch.from_numpy(rows)
            per.append(o4.dequant(rows) if L else np.zeros((0, Hkv, D)))
        caches.append(c)
        vals.append(per)
    return caches[0], caches[1], bt, vals[0], vals[1]

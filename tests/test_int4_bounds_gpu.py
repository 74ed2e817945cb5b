"""Decode over 4-bit caches against float64 with bounds that see a lost token or tile
(test_int4_bounds_cpu.py), through every way its tiles reach a warp (GB300 only)."""
import os
import random

import pytest
import torch

from int4_bounds import Case

pytestmark = pytest.mark.gpu

# 24 by default; PA_RANDOM_LONG runs more draws of the same seeded generator
N_LONG = int(os.environ.get("PA_RANDOM_LONG", "24"))
EDGES = (0, 1, 15, 16, 31, 32, 33, -1, -2, -33)


def shares(pa, c, splits=0, total_tokens=0):
    """Whether the call's splits share out their tails; (S, P)."""
    S, P = pa.plan(len(c.lens), c.Hq, c.Hkv, c.D, c.bs, max(c.lens), splits=splits, window=c.window,
                   total_tokens=total_tokens, kv_int4=True, rows=c.rows)
    return S > 1 and P * 2 * pa.int4_row_bytes(c.D) >= 512 << 10, (S, P)


def check(pa, c, calls=1, **kw):
    ref, tol = c.reference()
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(calls):      # the next call finds the counters as this one left them
        got = c.decode(pa, ws, **kw).double().cpu().numpy()
        assert pa.read_device_errors(ws) == 0
        assert not ws[:pa.PA_WORKSPACE_HEADER_BYTES].any()
        worst, norm = c.errors(got, ref, tol)
        assert worst <= 1 and norm <= 1, (worst, norm)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,lens,rows", [
    (8, 8, 128, 16, [512, 1, 33], 1), (32, 8, 128, 16, [1000, 37, 4097], 1), (24, 4, 256, 784, [500, 785, 3000], 1),
    (16, 1, 256, 33, [700, 5], 1), (12, 1, 128, 7, [63, 64, 65], 1), (6, 2, 128, 1, [130], 1),
    (32, 8, 128, 16, [2000, 4], 4), (8, 2, 128, 16, [900, 8], 8), (16, 2, 256, 784, [1700, 2], 2),
])
@pytest.mark.parametrize("heavy", [(), EDGES])
def test_shapes(cuda_lib, dtype, Hq, Hkv, D, bs, lens, rows, heavy):
    c = Case(lens, Hq, Hkv, D, bs, dtype, rows, seed=1, heavy=heavy)
    for splits in (0, 1, 3):
        check(cuda_lib, c, splits=splits)


@pytest.mark.parametrize("S", [1, 2, 3, 5, 8, 9, 40])
@pytest.mark.parametrize("D,bs", [(128, 16), (256, 100)])
def test_fixed_splits(cuda_lib, S, D, bs):
    P = cuda_lib.plan(4, 8, 2, D, bs, 2500, splits=S, kv_int4=True)[1]
    c = Case([2500, 1, 0, 777], 8, 2, D, bs, "f16", seed=2, heavy=EDGES + (P - 1, P, 2 * P - 1, 2 * P))
    check(cuda_lib, c, splits=S, deterministic=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,bs,S,longest,rows", [
    (4, 2, 128, 16, 2, 7000, 1),     # two splits in a cluster
    (4, 1, 128, 33, 3, 10100, 1),    # three
    (8, 2, 128, 16, 8, 27001, 1),    # eight
    (4, 1, 128, 16, 10, 36007, 1),   # a merge grid
    (8, 2, 128, 16, 2, 7111, 4),     # 16 columns
    (4, 1, 128, 7, 10, 35555, 8),    # 32 columns, a merge grid
    (6, 1, 256, 784, 2, 3500, 1), (3, 1, 256, 100, 8, 13600, 1), (3, 1, 256, 16, 11, 18500, 1),
    (6, 1, 256, 784, 2, 4001, 2), (6, 1, 256, 48, 10, 17777, 2),
])
def test_shared_tails(cuda_lib, dtype, Hq, Hkv, D, bs, S, longest, rows):
    # a long sequence with a ragged end, one that ends inside its first split, one that ends in
    # the second, an empty one; heavy tokens at both ends, where the static shares end and in the
    # tiles behind them that are shared out
    P = cuda_lib.plan(4, Hq, Hkv, D, bs, longest, splits=S, kv_int4=True, rows=rows)[1]
    Ps = P - P // 8 // 32 * 32
    heavy = EDGES + (Ps - 1, Ps, S * Ps - 1, S * Ps, S * Ps + 31, S * Ps + 32, -100)
    c = Case([longest, 50, P + 77, 0], Hq, Hkv, D, bs, dtype, rows, seed=3, heavy=heavy)
    ok, (splits, _) = shares(cuda_lib, c, S)
    assert ok and splits == S
    check(cuda_lib, c, calls=3, splits=S)
    check(cuda_lib, c, splits=S, deterministic=True)


@pytest.mark.parametrize("W", [1, 17, 1000])
def test_windows(cuda_lib, W):
    for Hq, Hkv, D, bs, dtype in ((8, 4, 128, 16, "bf16"), (6, 2, 256, 784, "f16"), (16, 1, 256, 100, "f16")):
        c = Case([1500, 999, 16, 1], Hq, Hkv, D, bs, dtype, window=W, seed=4, heavy=(-1, -W, -W - 1, -2))
        check(cuda_lib, c)
    c = Case([15000], 4, 1, 128, 16, "f16", window=9001, seed=5, heavy=(-1, -9001, -9002))
    assert shares(cuda_lib, c, 2)[0]
    check(cuda_lib, c, calls=2, splits=2)


@pytest.mark.parametrize("B,Hq,Hkv,D,bs,rows", [
    (32, 16, 8, 128, 16, 1), (50, 8, 4, 128, 16, 2), (200, 4, 2, 128, 16, 1), (256, 6, 2, 256, 48, 1),
    (41, 16, 4, 256, 784, 1), (24, 64, 8, 128, 16, 4),
])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_by_length(cuda_lib, B, Hq, Hkv, D, bs, rows, dtype):
    # unsplit, the longest sequences' CTAs first
    r = random.Random(B)
    lens = [r.randint(0, 200) for _ in range(B)]
    lens[B // 3], lens[B // 2], lens[-1] = 4000, 0, 3999
    c = Case(lens, Hq, Hkv, D, bs, dtype, rows, seed=6, heavy=(0, -1, 31))
    assert B * Hkv > 152 and sum(lens) < 7 * B * 4000 // 8
    check(cuda_lib, c, splits=1, total_tokens=sum(lens))


@pytest.mark.parametrize("B,Hq,Hkv,D,bs,longest", [
    (40, 8, 4, 128, 16, 300), (160, 1, 1, 128, 7, 2000), (30, 24, 6, 256, 33, 500), (90, 4, 2, 256, 784, 1900),
])
def test_short_ctas(cuda_lib, B, Hq, Hkv, D, bs, longest):
    r = random.Random(B)
    lens = [r.randint(0, longest) for _ in range(B)]
    lens[0], lens[1], lens[2] = longest, 0, 1
    check(cuda_lib, Case(lens, Hq, Hkv, D, bs, "f16", seed=7, heavy=(0, -1)))


@pytest.mark.parametrize("idx", range(N_LONG))
def test_random_long_contexts(cuda_lib, idx):
    r = random.Random(9000 + idx)
    D = r.choice([128, 256])
    rows = r.choice([1, 1, 2, 4])
    G = r.choice([g for g in (1, 2, 4, 6, 8) if g * rows <= (32 if D == 128 else 16)])
    Hkv, B = r.choice([1, 2]), r.randint(1, 3)
    lens = [int(2 ** r.uniform(6, 14.6)) for _ in range(B)]
    splits = r.choice([0, 2, 3, 8, 9])
    c = Case(lens, G * Hkv, Hkv, D, r.choice([1, 7, 16, 48, 784]), r.choice(["bf16", "f16"]), rows, seed=idx,
             heavy=tuple(r.randrange(max(lens)) for _ in range(8)) + (0, -1), k_scale=r.choice([1.0, 0.3]),
             v_scale=r.choice([1.0, 2.0]))
    check(cuda_lib, c, calls=2, splits=splits, total_tokens=r.choice([0, sum(lens)]))
